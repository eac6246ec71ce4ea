"""key_bounds' windows against enumeration."""
import pytest

from attention_forward_mode_b200 import key_bounds


def visible(Lk, p, causal=False, frame=0, window=0, documents=None):
    """The keys that a row at position p sees, by the rules one by one."""
    first, last = 0, Lk
    if documents is not None:
        own = [(a, b) for a, b in zip(documents, documents[1:]) if a <= p < b]
        if not own:
            return set()
        first, last = own[0]
    if p < 0 and frame:
        return set()
    seen = set(range(max(first, 0), min(last, Lk)))
    if causal:
        seen = {j for j in seen if j <= p}
    if frame:
        seen = {j for j in seen if (j - first) // frame <= (p - first) // frame}
    if window:
        seen = {j for j in seen if j > p - window and (frame or j <= p)}
    return seen


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=3), dict(window=100), dict(window=2, causal=True),
                                dict(window=2, frame=3), dict(window=5, frame=2), dict(window=2, documents=[0, 4, 9]),
                                dict(window=2, documents=[1, 3, 7], causal=True),
                                dict(window=4, documents=[0, 5, 5, 11], frame=3)], ids=str)
def test_windows_enumerated(kw):
    for Lq, Lk in ((7, 7), (4, 11), (11, 4), (1, 1)):
        begin, end = key_bounds(Lq, Lk, device="cpu", **kw)
        for i in range(Lq):
            seen = set(range(max(0, int(begin[i])), min(Lk, int(end[i]))))
            assert seen == visible(Lk, i + Lk - Lq, **kw), (Lq, Lk, i)


def test_a_window_and_a_prefix_are_no_interval():
    with pytest.raises(ValueError, match="interval"):
        key_bounds(8, 8, device="cpu", causal=True, prefix=3, window=2)
