"""The example that runs a stack of MXFP4 feed-forward blocks (prefill, decode, HIP graph)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,d,f,prefill,batch", [(2, 512, 1280, 130, 5), (1, 128, 128, 1, 1), (3, 1024, 640, 33, 64)])
def test_stack(layers, d, f, prefill, batch):
    from bf16_gemm_linear_amd import mxfp4_ffn

    got = mxfp4_ffn.main(["--layers", str(layers), "--d", str(d), "--f", str(f), "--prefill", str(prefill),
                          "--batch", str(batch)])  # compares the graph's replays with the calls
    # 4.25 bits a value against 16
    assert got["weight_bytes_mxfp4"] * 16 == got["weight_bytes_bf16"] * 4.25
    # A value between two codes is off by at most 1/4 of itself (between 4 and 6 by 1 of 5; to 8 by
    # 2 of 8), 1/8 rms; three products' operands make at most sqrt(6)/8 = 0.31 of a block's output,
    # to which the exact residual is added.
    for name in ("prefill", "decode"):
        assert got[name]["relative_error"] < 0.31, got
        assert got[name]["mxfp4_ms"] > 0
    assert got["decode"]["mxfp4_graph_ms"] > 0
