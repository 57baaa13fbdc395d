"""Host-side checks of the low-bit operators: pins of their fp64 definitions by
hand, and what the C ABI and the binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_gated_attention_b200 as sga
from oracle import lowbit
from sparse_gated_attention_b200 import build as sga_build


@pytest.fixture(scope="module")
def lib():
    sga_build.build()
    return sga.load_library()


# ----------------------------------------------------------------------------- the definitions, by hand
def test_e4m3_table():
    assert lowbit.E4M3[0x7E] == 448 and lowbit.E4M3[0x01] == 2.0 ** -9 and lowbit.E4M3[0x08] == 2.0 ** -6
    assert lowbit.E4M3[0x38] == 1 and lowbit.E4M3[0xB9] == -1.125 and np.isnan(lowbit.E4M3[0xFF])
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(lowbit.E4M3, want)


def test_quantize_by_hand():
    x = np.zeros((1, 130))
    x[0, :5] = [448, 17, 19, -0.001953125 / 2, 3.5]  # scale 1: ties 17 -> 16, 19 -> 20, half the least step -> 0
    x[0, 128:] = [450, -1]                            # the second block: scale 2
    codes, scale = lowbit.quantize_fp8(x)
    np.testing.assert_array_equal(scale, [[1, 2]])
    np.testing.assert_array_equal(lowbit.E4M3[codes][0, :5], [448, 16, 20, 0, 3.5])
    np.testing.assert_array_equal(lowbit.E4M3[codes][0, 128:], [224, -0.5])


def test_block_scaled_by_hand():
    codes = np.full((129, 130), 0x38, dtype=np.uint8)  # ones
    v = lowbit.block_scaled(codes, np.array([[2.0, 3.0], [5.0, 7.0]]), 128)
    assert v[0, 0] == 2 and v[127, 128] == 3 and v[128, 127] == 5 and v[128, 129] == 7


def test_kv4_by_hand():
    row = np.zeros((1, 576))
    row[0, :4] = [12, -1, 0.5, -0.5]  # scale 2: -1 / 2 -> -0.5, 0.25 ties to 0
    row[0, 16] = 1e6                  # saturates: scale 448, code 6
    row[0, 512:514] = [1.5, -2]
    code, scale, rope = lowbit.kv4_pack(row)
    assert list(code[0, :4]) == [7, 9, 0, 8] and lowbit.E4M3[scale[0, 0]] == 2
    assert code[0, 16] == 7 and lowbit.E4M3[scale[0, 1]] == 448
    packed = np.zeros((1, 416), dtype=np.uint8)
    packed[0, 0], packed[0, 1], packed[0, 8] = 7 | (9 << 4), 0 | (8 << 4), 7
    packed[0, 256:258] = scale[0, :2]
    packed[0, 288:292] = [0xC0, 0x3F, 0x00, 0xC0]
    v = lowbit.kv4_values(packed)[0]
    np.testing.assert_array_equal(v[:4], [12, -1, 0, 0])
    np.testing.assert_array_equal([v[16], v[512], v[513]], [2688, 1.5, -2])


def test_attend_by_hand():
    """Two rows with equal logits average; a third is not selected; one head is gated by one half."""
    packed = np.zeros((1, 3, 416), dtype=np.uint8)
    packed[0, 0, 0], packed[0, 1, 0], packed[0, 2, 0] = 2, 4, 7  # dim 0: 1, 2, 6
    packed[0, :, 256] = 0x38
    q = np.zeros((1, 1, 2, 576))
    idx = np.array([[[1, -1, 0]]])
    out = lowbit.attend_kv4(q, packed, idx, np.array([[[0.0, 100.0]]]))[0]
    np.testing.assert_allclose(out[0, 0, :, 0], [0.75, 1.5])
    q[0, 0, 1, 0] = np.log(3.0) * 192 ** 0.5  # row 1's logit is larger by log 3: weights 3/4 and 1/4
    out = lowbit.attend_kv4(q, packed, idx, None)[0]
    np.testing.assert_allclose(out[0, 0, :, 0], [1.5, 1.75])


# ----------------------------------------------------------------------------- refusals
P = ctypes.c_void_p
GOOD, ODD, WS = P(0x100000), P(0x100002), P(0x20000000)


def test_kv4_calls_refuse_bad_arguments(lib):
    d = sga.make_dims(2, 3, 1000)
    r = ctypes.byref(d)
    assert lib.sga_kv4_append(r, None, GOOD, GOOD, WS, 256, None) == 1
    assert lib.sga_kv4_append(r, ODD, GOOD, GOOD, WS, 256, None) == 1
    assert lib.sga_kv4_append(r, GOOD, GOOD, ODD, WS, 256, None) == 1
    assert lib.sga_kv4_append(r, GOOD, GOOD, GOOD, None, 256, None) == 3
    assert lib.sga_kv4_append(r, GOOD, GOOD, GOOD, P(0x20000010), 256, None) == 3
    assert lib.sga_kv4_append(r, GOOD, GOOD, GOOD, WS, 255, None) == 3
    assert lib.sga_kv4_append(None, GOOD, GOOD, GOOD, WS, 256, None) == 1
    half = P(0x100010)  # a cache row is read 32 bytes at a time
    assert lib.sga_kv4_append(r, GOOD, GOOD, half, WS, 256, None) == 1
    assert lib.sga_kv4_read(r, half, GOOD, GOOD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, half, GOOD, None, GOOD, WS, 256, None) == 1
    assert lib.sga_kv4_read(r, GOOD, None, GOOD, WS, 256, None) == 1
    assert lib.sga_kv4_read(r, GOOD, GOOD, ODD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, None, GOOD, None, GOOD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, GOOD, P(0x100004), None, GOOD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, GOOD, GOOD, P(0x100001), GOOD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, GOOD, GOOD, None, GOOD, WS, 128, None) == 3
    a = (GOOD,) * 4
    assert lib.sga_forward_kv4(r, *a, None, None, GOOD, None, GOOD, WS, 1 << 30, None) == 1
    assert lib.sga_forward_kv4(r, *a, GOOD, None, GOOD, None, None, WS, 1 << 30, None) == 1
    assert lib.sga_forward_kv4(r, *a, GOOD, None, GOOD, None, P(0x100008), WS, 1 << 30, None) == 1
    assert lib.sga_forward_kv4(r, *a, GOOD, None, GOOD, None, GOOD, WS, 4096, None) == 3


@pytest.mark.parametrize("dims", [(0, 1, 100, 64), (1, 0, 100, 64), (1, 1, 0, 64), (1, 1, (1 << 30) + 1, 64),
                                  (3, 1, 1 << 30, 64), (1 << 16, 1 << 10, 10, 64)])
def test_kv4_calls_refuse_bad_sizes(lib, dims):
    d = sga.make_dims(*dims)
    r = ctypes.byref(d)
    assert lib.sga_kv4_append(r, GOOD, GOOD, GOOD, WS, 256, None) == 1
    assert lib.sga_kv4_read(r, GOOD, GOOD, GOOD, WS, 256, None) == 1
    assert lib.sga_sparse_mla_attend_kv4(r, GOOD, GOOD, GOOD, None, GOOD, WS, 256, None) == 1


@pytest.mark.parametrize("top_k", [0, 63, 65, 2112, -64])
def test_attend_kv4_refuses_bad_top_k(lib, top_k):
    d = sga.make_dims(1, 1, 1000, top_k)
    assert lib.sga_sparse_mla_attend_kv4(ctypes.byref(d), GOOD, GOOD, GOOD, None, GOOD, WS, 256, None) == 1


def test_quantize_refuses_bad_arguments(lib):
    for rows, cols in [(0, 16), (1, 0), (1, 15), (1, 24), (-1, 16)]:
        assert lib.sga_quantize_fp8(rows, cols, GOOD, GOOD, GOOD, None) == 1
    assert lib.sga_quantize_fp8(1, 2**31 - 16, GOOD, GOOD, GOOD, None) == 1
    assert lib.sga_quantize_fp8(1, 16, ODD, GOOD, GOOD, None) == 1
    assert lib.sga_quantize_fp8(1, 16, GOOD, P(0x100008), GOOD, None) == 1
    assert lib.sga_quantize_fp8(1, 16, GOOD, GOOD, None, None) == 1
    assert lib.sga_quantize_fp8(1, 16, GOOD, GOOD, ODD, None) == 1


@pytest.mark.parametrize("rows,cols", [(2**30 + 1, 16), (2**31 - 1, 128), (2**29 + 1, 144), (2**20, 2**18)])
def test_quantize_refuses_more_than_2_to_30_scales(lib, rows, cols):
    assert lib.sga_quantize_fp8(rows, cols, GOOD, GOOD, GOOD, None) == 1


def test_product_refuses_bad_arguments(lib):
    def call(n=4, m=5, k=32, x=GOOD, xs=GOOD, w=GOOD, wsc=GOOD, y=GOOD, t=0, ws=WS, nbytes=256):
        return lib.sga_gemm_fp8(n, m, k, x, xs, w, wsc, y, t, ws, nbytes, None)

    top = 2**31 - 1
    for bad in [dict(n=0), dict(m=0), dict(k=0), dict(k=24), dict(n=-3), dict(n=top), dict(m=top), dict(k=top - 15), dict(t=2), dict(x=None), dict(x=ODD),
                dict(w=ODD), dict(xs=ODD), dict(wsc=None), dict(y=None), dict(y=ODD), dict(y=P(0x100001), t=1)]:
        assert call(**bad) == 1, bad
    for bad in [dict(ws=None), dict(ws=P(0x20000010)), dict(nbytes=255)]:
        assert call(**bad) == 3, bad


def test_binding_refuses_cpu_tensors_and_wrong_types():
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.quantize_fp8(torch.zeros((2, 32), dtype=bf))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.gemm_fp8(torch.zeros((2, 32), dtype=u8), torch.zeros((2, 1)), torch.zeros((4, 32), dtype=u8),
                     torch.zeros((1, 1)))
    with pytest.raises(ValueError, match=r"expected \[..., K\]"):
        sga.gemm_fp8(torch.zeros((2, 32), dtype=u8), None, torch.zeros(32, dtype=u8), None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.kv4_append(torch.zeros((1, 1, 576), dtype=bf), torch.zeros((1, 1), dtype=i32),
                       torch.zeros((1, 8, 416), dtype=u8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.kv4_read(torch.zeros((1, 8, 416), dtype=u8), torch.zeros((1, 1), dtype=i32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.sparse_mla_attend_kv4(torch.zeros((1, 1, 64, 576), dtype=bf), torch.zeros((1, 8, 416), dtype=u8),
                                  torch.zeros((1, 1, 64), dtype=i32))


def test_binding_refuses_extents_past_32_bits(monkeypatch):
    """The library takes 32-bit extents: a longer one is refused, not cut to its low bits (the first tensor here would
    be quantised in its first 16 channels only)."""
    from sparse_gated_attention_b200 import _binding

    def big(*shape, dtype=torch.uint8):
        return torch.empty(shape, dtype=dtype, device="meta")

    monkeypatch.setattr(_binding, "_need", lambda t, *a: t)
    monkeypatch.setattr(_binding, "_one_device", lambda *t: None)
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    with pytest.raises(ValueError, match="2\\^31"):
        sga.quantize_fp8(big(1, 2 ** 32 + 16, dtype=bf))
    with pytest.raises(ValueError, match="2\\^31"):
        sga.quantize_fp8(big(2 ** 32 + 1, 16, dtype=bf))
    for x, w in ((big(1, 16), big(2 ** 32 + 5, 16)), (big(1, 2 ** 32 + 16), big(3, 2 ** 32 + 16)),
                 (big(2 ** 31, 2, 16), big(3, 16))):
        with pytest.raises(ValueError, match="2\\^31"):
            sga.gemm_fp8(x, big(1, dtype=f32), w, big(1, dtype=f32))
    row, q, cache = big(1, 1, 576, dtype=bf), big(1, 1, 64, 576, dtype=bf), big(1, 2 ** 32 + 8, 416)
    pos, ws = big(1, 1, dtype=i32), big(256)
    with pytest.raises(ValueError, match="2\\^31"):
        sga.kv4_append(row, pos, cache, ws=ws)
    with pytest.raises(ValueError, match="2\\^31"):
        sga.kv4_read(cache, pos, row, ws=ws)
    with pytest.raises(ValueError, match="2\\^31"):
        sga.sparse_mla_attend_kv4(q, cache, big(1, 1, 64, dtype=i32), out=q, ws=ws)
    with pytest.raises(ValueError, match="2\\^31"):
        sga.sparse_mla_attend_kv4(q, big(1, 8, 416), big(1, 1, 2 ** 32 + 64, dtype=i32), out=q, ws=ws)
    for extents in ((2 ** 32 + 1, 1, 1), (1, 2 ** 31, 1), (1, 1, 2 ** 32 + 5), (1, 1, 5, 2 ** 32 + 64),
                    (5 - 2 ** 32, 1, 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            sga.make_dims(*extents)
    assert sga.make_dims(1, 2, 3, 2 ** 31 - 1).top_k == 2 ** 31 - 1


def _fp8_weights(d_model=7168, q_rank=1536, **bad):
    names = ("w_hq", "w_hq_scale", "w_cq", "w_cq_scale", "w_o", "w_o_scale", "w_uk", "w_uv")
    return sga.LayerFp8Weights(d_model, q_rank, *(bad.get(n, 0x300000 + 0x100000 * i) for i, n in enumerate(names)))


def test_layer_fp8kv4_workspace_and_refusals(lib):
    d = sga.make_dims(32, 1, 131072)
    size = sga.layer_fp8kv4_workspace_size(d, _fp8_weights())
    assert size >= sga.workspace_size(d) + 32 * 4 * (20608 + 1536 + 832)
    r, big = ctypes.byref(d), 1 << 40

    def call(W=_fp8_weights(), dims=r, h=GOOD, pos=GOOD, kv4=GOOD, k=GOOD, idx=None, y=GOOD, ws=WS, nbytes=256):
        return lib.sga_layer_forward_fp8kv4(dims, ctypes.byref(W), h, pos, kv4, k, idx, y, ws, nbytes, None)

    for W in (_fp8_weights(d_model=7160), _fp8_weights(q_rank=1528), _fp8_weights(d_model=0), _fp8_weights(w_hq=0),
              _fp8_weights(w_cq=0x400008), _fp8_weights(w_o_scale=0), _fp8_weights(w_hq_scale=0x500002),
              _fp8_weights(w_uk=2), _fp8_weights(w_uv=0)):
        assert call(W=W) == 1
    for bad in (dict(h=ODD), dict(pos=None), dict(kv4=P(0x100008)), dict(k=ODD), dict(idx=ODD), dict(y=None)):
        assert call(**bad) == 1, bad
    assert call(dims=ctypes.byref(sga.make_dims(1, 1, 100, 65))) == 1
    for bad in (dict(ws=None), dict(ws=P(0x20000010)), dict(nbytes=size - 1)):
        assert call(**bad) == 3, bad
    out = ctypes.c_size_t(0)
    assert lib.sga_layer_fp8kv4_workspace_size(r, None, ctypes.byref(out)) == 1
    assert lib.sga_layer_fp8kv4_workspace_size(r, ctypes.byref(_fp8_weights()), None) == 1


def test_layer_sizes_past_2_to_30_are_refused(lib):
    """A width near 2^31 made the size checks wrap, and gave a workspace size that had wrapped as well."""
    out = ctypes.c_size_t(0)
    d = ctypes.byref(sga.make_dims(1, 1, 100))
    top = 1 << 30
    for width in (top + 16, 2 ** 31 - 1024, 2 ** 31 - 16):
        for bad in (dict(d_model=width), dict(q_rank=width)):
            W = _fp8_weights(**bad)
            assert lib.sga_layer_fp8kv4_workspace_size(d, ctypes.byref(W), ctypes.byref(out)) == 1, bad
            assert lib.sga_layer_forward_fp8kv4(d, ctypes.byref(W), GOOD, GOOD, GOOD, GOOD, None, GOOD, WS, 1 << 60,
                                                None) == 1, bad
    assert lib.sga_layer_fp8kv4_workspace_size(d, ctypes.byref(_fp8_weights(q_rank=top)), ctypes.byref(out)) == 0
    assert out.value > top * 7  # codes, g1 and c_q of one token
