"""Rotary positions and the paged append on the host (no GPU): argument checks
of attn_rope and attn_paged_append before any CUDA call, and the frequency
tables with their long-context scalings."""
import math

import pytest

from tiled_attention_17_b200 import rope


@pytest.fixture(scope="module")
def lib():
    from tiled_attention_17_b200 import binding, build
    build.build()
    return binding


def test_rope_validation(lib):
    a = 256   # 16-byte-aligned non-null value: rejected before use

    def call(**kw):
        g = dict(x=a, y=2 * a, pos=a, f=a, B=1, H=2, N=8, d=128, r=64, il=0, inv=0, amp=1.0, xb=0, xh=128, xn=256,
                 yb=0, yh=1024, yn=128, pb=0)
        g.update(kw)
        return lib.STATUS_NAMES[lib.attn_rope(g["x"], g["y"], g["pos"], g["f"], g["B"], g["H"], g["N"], g["d"], g["r"],
                                              g["il"], g["inv"], g["amp"], g["xb"], g["xh"], g["xn"], g["yb"], g["yh"],
                                              g["yn"], g["pb"], stream=0, check=False)]

    assert call(B=-1) == "TA_ERR_INVALID_ARG"
    assert call(d=96) == "TA_ERR_UNSUPPORTED"
    assert call(r=24) == "TA_ERR_UNSUPPORTED"              # halves that are not whole 16-byte vectors
    assert call(r=144) == "TA_ERR_INVALID_ARG"             # more than the head
    assert call(r=-16) == "TA_ERR_INVALID_ARG"
    assert call(il=2) == "TA_ERR_INVALID_ARG"
    assert call(inv=2) == "TA_ERR_INVALID_ARG"
    assert call(amp=float("nan")) == "TA_ERR_INVALID_ARG"
    assert call(f=None) == "TA_ERR_INVALID_ARG"
    assert call(f=a + 4) == "TA_ERR_INVALID_ARG"           # fp64 alignment
    assert call(x=None) == "TA_ERR_INVALID_ARG"
    assert call(x=a + 8) == "TA_ERR_INVALID_ARG"
    assert call(y=a + 2) == "TA_ERR_INVALID_ARG"
    assert call(pos=a + 2) == "TA_ERR_INVALID_ARG"
    assert call(xn=132) == "TA_ERR_INVALID_ARG"            # rows off the 16-byte grid
    assert call(yh=0) == "TA_ERR_INVALID_ARG"              # two heads on one row
    assert call(y=a) == "TA_ERR_INVALID_ARG"               # in place with other strides
    assert call(H=65536) == "TA_ERR_UNSUPPORTED"
    assert call(B=65536, N=65536, yb=8) == "TA_ERR_UNSUPPORTED"
    for empty in (dict(B=0), dict(H=0), dict(N=0)):
        assert call(**empty) == "TA_OK"


def test_append_validation(lib):
    a = 256

    def call(**kw):
        g = dict(q=a, k=a, v=a, qo=a, kc=a, vc=a, bt=a, cu=a, sl=a, pos=None, f=a, ps=16, S=2, T=9, Hq=4, Hkv=2,
                 d=128, mp=8, P=20, r=128, il=0, amp=1.0, qs=(512, 128), ks=(256, 128), vs=(256, 128))
        g.update(kw)
        return lib.STATUS_NAMES[lib.attn_paged_append(
            g["q"], g["k"], g["v"], g["qo"], g["kc"], g["vc"], g["bt"], g["cu"], g["sl"], g["pos"], g["f"], g["ps"],
            g["S"], g["T"], g["Hq"], g["Hkv"], g["d"], g["mp"], g["P"], g["r"], g["il"], g["amp"], *g["qs"],
            *g["ks"], *g["vs"], stream=0, check=False)]

    assert call(ps=12) == "TA_ERR_UNSUPPORTED"
    assert call(d=80, r=64) == "TA_ERR_UNSUPPORTED"
    assert call(r=40) == "TA_ERR_UNSUPPORTED"
    assert call(r=256) == "TA_ERR_INVALID_ARG"
    assert call(mp=1 << 27) == "TA_ERR_UNSUPPORTED"        # 2^31 tokens
    assert call(Hkv=0) == "TA_ERR_INVALID_ARG"
    assert call(Hq=0) == "TA_ERR_INVALID_ARG"
    assert call(S=-1) == "TA_ERR_INVALID_ARG"
    assert call(cu=None) == "TA_ERR_INVALID_ARG"           # one token per sequence: total == num_seqs
    assert call(qo=None) == "TA_ERR_INVALID_ARG"
    assert call(k=None) == "TA_ERR_INVALID_ARG"
    assert call(kc=a + 8) == "TA_ERR_INVALID_ARG"
    assert call(sl=a + 2) == "TA_ERR_INVALID_ARG"
    assert call(ks=(260, 128)) == "TA_ERR_INVALID_ARG"
    assert call(qs=(1024, 128)) == "TA_ERR_INVALID_ARG"    # in place, but q's rows are not q_out's
    assert call(f=None) == "TA_ERR_INVALID_ARG"
    assert call(amp=float("inf")) == "TA_ERR_INVALID_ARG"
    assert call(T=(1 << 30) + 1) == "TA_ERR_UNSUPPORTED"
    assert call(T=0) == "TA_OK"
    assert call(S=0) == "TA_OK"


def test_plain_and_scaled_frequencies():
    f, amp = rope.frequency_list(8, 10000.0)
    assert amp == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    g, amp = rope.frequency_list(8, 10000.0, {"type": "linear", "factor": 4.0})
    assert amp == 1.0 and g == pytest.approx([x / 4 for x in f], rel=1e-15)
    # a larger base keeps the fastest pair and divides the slowest by the factor
    g, amp = rope.frequency_list(64, 10000.0, {"type": "ntk", "factor": 8.0})
    slow = 10000.0 ** (-62 / 64)
    assert g[0] == 1.0 and g[-1] == pytest.approx(slow / 8, rel=1e-12)


@pytest.mark.parametrize("kind", ["yarn", "wavelength"])
def test_banded_scalings_keep_fast_pairs_and_divide_slow_ones(kind):
    trained, factor = 4096, 16.0
    f, _ = rope.frequency_list(128)
    g, amp = rope.frequency_list(128, scaling={"type": kind, "factor": factor, "trained_length": trained})
    assert amp == pytest.approx(0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)
    most = 33.0 if kind == "yarn" else 4.0
    for a, b in zip(f, g):
        turns = trained * a / (2 * math.pi)
        assert a / factor * (1 - 1e-12) <= b <= a * (1 + 1e-12)
        if turns >= most * 1.5:
            assert b == pytest.approx(a, rel=1e-12)
        if turns <= 0.6:
            assert b == pytest.approx(a / factor, rel=1e-12)
    assert all(x >= y for x, y in zip(g, g[1:]))


@pytest.mark.parametrize("args", [
    (7,), (0,), (8, 1.0), (8, float("nan")), (8, 1e4, {"type": "other", "factor": 2.0}), (8, 1e4, {"type": "linear"}),
    (8, 1e4, {"type": "linear", "factor": 0.5}), (8, 1e4, {"type": "linear", "factor": 2.0, "beta_fast": 3}),
    (8, 1e4, {"type": "yarn", "factor": 2.0}), (2, 1e4, {"type": "ntk", "factor": 2.0}),
    (8, 1e4, {"type": "yarn", "factor": 2.0, "trained_length": 100, "beta_fast": 1.0, "beta_slow": 2.0}),
    (8, 1e4, {"type": "wavelength", "factor": 2.0, "trained_length": -1}),
])
def test_frequency_refusals(args):
    with pytest.raises(ValueError):
        rope.frequency_list(*args)


def test_yarn_ramp_at_known_pairs():
    # trained 4096, base 10^4, 64 pairs: 32 turns fall at pair 64 ln(4096 / 64 pi) / ln 10^4 = 20.94, one turn at
    # 64 ln(4096 / 2 pi) / ln 10^4 = 45.03, so the ramp goes from pair 20 to pair 46
    f, _ = rope.frequency_list(128)
    g, _ = rope.frequency_list(128, scaling={"type": "yarn", "factor": 16.0, "trained_length": 4096})
    for pair, kept in ((0, 1.0), (20, 1.0), (21, 25 / 26), (26, 20 / 26), (33, 0.5), (45, 1 / 26), (46, 0.0), (63, 0.0)):
        assert g[pair] == pytest.approx(f[pair] * (kept + (1 - kept) / 16), rel=1e-12), pair
    # other betas: 16 turns at 25.76, 2 turns at 40.21
    g, _ = rope.frequency_list(128, scaling={"type": "yarn", "factor": 4.0, "trained_length": 4096, "beta_fast": 16.0,
                                             "beta_slow": 2.0})
    for pair, kept in ((25, 1.0), (33, 0.5), (37, 0.25), (41, 0.0)):
        assert g[pair] == pytest.approx(f[pair] * (kept + (1 - kept) / 4), rel=1e-12), pair


@pytest.mark.parametrize("turns,kept", [(0.5, 0.0), (1.0, 0.0), (1.75, 0.25), (2.5, 0.5), (3.25, 0.75), (4.0, 1.0), (9.0, 1.0)])
def test_wavelength_ramp_at_known_turns(turns, kept):
    # pair 1 of 4 at base 10^4 turns by 0.1 a position: `turns` over this trained length; the ramp is linear in the turns
    trained = turns * 2 * math.pi / 0.1
    g, amp = rope.frequency_list(8, 10000.0, {"type": "wavelength", "factor": 8.0, "trained_length": trained})
    assert amp == 1.0 and g[1] == pytest.approx(0.1 * (kept + (1 - kept) / 8), rel=1e-12)
    # other ends of the ramp
    g, _ = rope.frequency_list(8, 10000.0, {"type": "wavelength", "factor": 8.0, "trained_length": trained, "low_turns": 0.5,
                                            "high_turns": 8.5})
    share = min(max((turns - 0.5) / 8, 0.0), 1.0)
    assert g[1] == pytest.approx(0.1 * (share + (1 - share) / 8), rel=1e-12)
