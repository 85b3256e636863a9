"""The rotary frequencies between the bands, where the two ways to mix them differ: linear in the turns that a pair
makes within the original length, and linear in the pair's index (what models with YaRN in their configuration are
run with).  Written from the formulas, in FP64; powers, logarithms and divisions are good to 2^-48 here."""
import math

import pytest


@pytest.fixture(scope="module")
def Q():
    import moe_qw_repack_gb300.qw as q
    return q


CASES = [(1e4, 128, 16.0, 4096.0, 1.0, 32.0), (1e6, 128, 4.0, 32768.0, 1.0, 32.0), (1e4, 64, 40.0, 4096.0, 1.0, 32.0),
         (5e5, 128, 8.0, 8192.0, 1.0, 4.0), (1e4, 96, 2.5, 2048.0, 0.5, 20.0), (1.5e5, 64, 32.0, 4096.0, 1.0, 32.0),
         (1e4, 2, 8.0, 4096.0, 1.0, 32.0), (1e4, 4, 8.0, 4096.0, 1.0, 32.0), (1e4, 256, 1.0, 8192.0, 1.0, 32.0)]


def by_turns(base, rot, factor, original, low, high):
    out = []
    for j in range(rot // 2):
        f = base ** (-2 * j / rot)
        share = (original * f / (2 * math.pi) - low) / (high - low)
        share = min(1.0, max(0.0, share))
        out.append(share * f + (1 - share) * f / factor)
    return out


def by_index(base, rot, factor, original, low, high):
    def pair_of(turns):  # base^(-2 j / rot) original / (2 pi) = turns, solved for j
        return rot / 2 * math.log(original / (2 * math.pi * turns), base)
    first = max(math.floor(pair_of(high)), 0)
    last = min(math.ceil(pair_of(low)), rot - 1)
    out = []
    for j in range(rot // 2):
        f = base ** (-2 * j / rot)
        if j <= first:
            stretch = 0.0
        elif j >= last:
            stretch = 1.0
        else:
            stretch = (j - first) / (last - first)
        out.append(stretch * f / factor + (1 - stretch) * f)
    return out


def close(got, want):
    return len(got) == len(want) and all(abs(g - w) <= 2.0 ** -48 * w for g, w in zip(got.tolist(), want))


@pytest.mark.parametrize("case", CASES)
def test_linear_in_turns(Q, case):
    base, rot, factor, original, low, high = case
    for method, scale in ((Q.QW_ROPE_YARN, 0.1 * math.log(factor) + 1), (Q.QW_ROPE_BANDS, 1.0)):
        f, s = Q.qw_rope_frequencies(method, base, rot, factor, original, low, high)
        assert close(f, by_turns(*case))
        assert abs(s - scale) <= 2.0 ** -24 * scale


@pytest.mark.parametrize("case", CASES)
def test_linear_in_the_pair_index(Q, case):
    base, rot, factor, original, low, high = case
    f, s = Q.qw_rope_frequencies(Q.QW_ROPE_YARN_INDEX, base, rot, factor, original, low, high)
    assert close(f, by_index(*case))
    assert abs(s - (0.1 * math.log(factor) + 1)) <= 2.0 ** -24 * s


def test_the_two_differ_between_the_bands_only(Q):
    """Base 10^4, 128 values, 16 times 4096: pairs 21 to 45 are mixed.  Pair 32 turns 6.5 times; by turns it keeps
    5.5 / 31 of its frequency, by index (46 - 32) / (46 - 20)."""
    args = (1e4, 128, 16.0, 4096.0, 1.0, 32.0)
    t, _ = Q.qw_rope_frequencies(Q.QW_ROPE_YARN, *args)
    i, _ = Q.qw_rope_frequencies(Q.QW_ROPE_YARN_INDEX, *args)
    ratio = (i / t).tolist()
    assert all(r == 1.0 for r in ratio[:21] + ratio[46:])
    assert 2.4 < ratio[32] < 2.6 and 2.9 < ratio[36] < 3.1


def test_bands_outside_the_pairs(Q):
    """An original length in which no pair makes `high` turns, one in which all do, and a low of no turns: whatever
    is mixed lies between the stretched frequency and the kept one, and slower pairs are stretched no less."""
    for original, low, high in ((100.0, 1.0, 32.0), (1e12, 1.0, 32.0), (4096.0, 0.0, 32.0), (3.0, 1.0, 2.0),
                                (4096.0, 31.9, 32.0)):
        f, _ = Q.qw_rope_frequencies(Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0, original, low, high)
        kept = [v / 1e4 ** (-2 * j / 64) for j, v in enumerate(f.tolist())]
        assert all(0.125 * (1 - 1e-12) <= k <= 1 + 1e-12 for k in kept)
        assert all(b <= a + 1e-12 for a, b in zip(kept, kept[1:]))
    assert all(abs(k - 1) < 1e-12 for k in [v / 1e4 ** (-2 * j / 64) for j, v in enumerate(
        Q.qw_rope_frequencies(Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0, 1e12, 1.0, 32.0)[0].tolist())])


def test_refusals(Q):
    for args in [(Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0), (Q.QW_ROPE_YARN_INDEX, 1e4, 64, 0.5, 4096.0),
                 (Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0, 4096.0, 4.0, 4.0),
                 (Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0, 4096.0, -1.0, 4.0),
                 (Q.QW_ROPE_YARN_INDEX, 1e4, 64, 8.0, float("nan")), (6, 1e4, 64, 8.0, 4096.0)]:
        with pytest.raises(Q.QwError):
            Q.qw_rope_frequencies(*args)
