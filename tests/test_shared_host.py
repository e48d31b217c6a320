"""attn_paged_decode_shared on the host (no GPU): argument checks before any
CUDA call, and the workspace size."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from tiled_attention_17_b200 import binding, build
    build.build()
    return binding


def test_shared_validation(lib):
    a = 256
    ws = lib.attn_paged_decode_shared_workspace_size(4, 2, 8, 2, 128)

    def call(**kw):
        g = dict(q=a, kc=a, vc=a, bt=a, sl=a, go=a, pl=a, ps=16, S=4, NG=2, own=100, Hq=8, Hkv=2, d=128, mp=64, P=100,
                 scale=0.1, o=a, lse=None, ws=a, wsb=ws)
        g.update(kw)
        return lib.STATUS_NAMES[lib.attn_paged_decode_shared(
            g["q"], g["kc"], g["vc"], g["bt"], g["sl"], g["go"], g["pl"], g["ps"], g["S"], g["NG"], g["own"], g["Hq"],
            g["Hkv"], g["d"], g["mp"], g["P"], g["scale"], g["o"], g["lse"], g["ws"], g["wsb"], stream=0, check=False)]

    assert call(ps=12) == "TA_ERR_UNSUPPORTED"
    assert call(d=80) == "TA_ERR_UNSUPPORTED"
    assert call(Hq=6, Hkv=4) == "TA_ERR_INVALID_ARG"
    assert call(Hq=24, Hkv=2) == "TA_ERR_UNSUPPORTED"       # groups of 12 heads
    assert call(NG=-1) == "TA_ERR_INVALID_ARG"
    assert call(NG=65536) == "TA_ERR_UNSUPPORTED"
    assert call(own=-1) == "TA_ERR_INVALID_ARG"
    assert call(own=64 * 16 + 1) == "TA_ERR_INVALID_ARG"    # more than the table holds
    assert call(mp=1 << 27) == "TA_ERR_UNSUPPORTED"
    assert call(P=1 << 30, Hkv=2) == "TA_ERR_UNSUPPORTED"   # (page, head) blocks past a 32-bit coordinate
    assert call(scale=float("nan")) == "TA_ERR_UNSUPPORTED"
    assert call(go=None) == "TA_ERR_INVALID_ARG"
    assert call(pl=a + 2) == "TA_ERR_INVALID_ARG"
    assert call(q=a + 8) == "TA_ERR_INVALID_ARG"
    assert call(ws=a + 16) == "TA_ERR_INVALID_ARG"
    assert call(wsb=ws - 1) == "TA_ERR_INVALID_ARG"
    assert "workspace" in lib.ta_last_error()
    assert call(S=0) == "TA_OK"


def test_shared_workspace_size(lib):
    size = lib.attn_paged_decode_shared_workspace_size
    one = size(64, 1, 32, 8, 128)
    assert one % 256 == 0
    # one 256-row block per KV head and (148 SMs) one more per CTA, 128 KB each; two partials of
    # 4 rows for every sequence and KV head
    assert one >= (8 + 148) * 256 * 128 * 4 + 64 * 8 * 2 * 4 * 128 * 4
    assert size(64, 0, 32, 8, 128) < one - 148 * 256 * 128 * 4    # no groups: no prefix partials
    assert size(64, 1, 30, 8, 128) == 0
    assert size(64, 1, 32, 8, 96) == 0
    assert size(65536, 1, 32, 8, 128) == 0
    assert size(64, 65536, 32, 8, 128) == 0
    assert size(64, -1, 32, 8, 128) == 0


def test_stream_of_another_device_is_refused():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from tiled_attention_17_b200 import binding
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        binding._scope(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)))
