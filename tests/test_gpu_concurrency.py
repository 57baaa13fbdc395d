"""Concurrent calls on distinct workspaces.

The ABI allows calls on distinct workspaces from several host threads and
streams at once.  Two threads, each with its own stream, workspace and inputs,
run sga_forward twenty times while the other does the same, so their kernels
(persistent indexers, cluster top-k and attention) share the GPU.  Every
result must equal the oracle's (indices bit-exact, outputs within the path's
tolerance) and repeat bit for bit from call to call."""
import threading
import time

import numpy as np
import pytest
import torch

import oracle
import sparse_gated_attention_b200 as sga
from sparse_gated_attention_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_gated_attention_b200 import build
    build.build()
    sga.load_library()
    oracle.build()


def test_forward_from_two_threads_on_two_streams():
    cases = [synth.custom(batch=3, n_q=1, ctx=9000, first_pos=8999),
             synth.custom(batch=2, n_q=1, ctx=20000, first_pos=19999)]
    xs = [synth.make_inputs(wl, device="cuda", seed=20 + i) for i, wl in enumerate(cases)]
    wants = [oracle.forward(x["q_idx"], x["w"], x["k_idx"], x["q"], x["kv"], x["gate"], x["q_pos"].cpu())
             for x in xs]
    results = [[] for _ in cases]
    errors = []
    start = threading.Barrier(len(cases))

    def worker(i):
        try:
            wl, x = cases[i], xs[i]
            stream = torch.cuda.Stream()
            ws = sga.alloc_workspace(sga.make_dims(wl.batch, 1, wl.ctx), sga.OP_FORWARD)
            torch.cuda.synchronize()
            start.wait()
            outs = []
            with torch.cuda.stream(stream):
                for _ in range(20):
                    outs.append(sga.forward(x["q_idx"], x["w"], x["k_idx"], x["q"], x["kv"], x["gate"], x["q_pos"],
                                            ws=ws, stream=stream))
            stream.synchronize()
            if sga.device_status(ws, stream) != 0:
                errors.append((i, "device status"))
            results[i] = [(idx.cpu().numpy(), out.cpu().numpy()) for idx, out in outs]
        except Exception as exc:  # reported below, with the thread's index
            errors.append((i, repr(exc)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i, (want_idx, want_out) in enumerate(wants):
        assert len(results[i]) == 20
        idx0, out0 = results[i][0]
        np.testing.assert_array_equal(idx0, want_idx)
        err = out0.astype(np.float64) - want_out
        assert np.linalg.norm(err) / np.linalg.norm(want_out) <= 1e-3 and np.abs(err).max() <= 1e-2
        for idx, out in results[i][1:]:
            assert np.array_equal(idx, idx0) and np.array_equal(out, out0)


def _calls():
    """Every call of the binding that makes outputs or a workspace itself: name -> call(stream), a fresh result."""
    g = torch.Generator(device="cuda").manual_seed(40)
    wl = synth.custom(batch=2, n_q=1, ctx=3000, first_pos=2999)
    x = synth.make_inputs(wl, device="cuda", seed=41)
    B, T, L = 2, 1, 3000
    path = (x["q_idx"], x["w"], x["k_idx"], x["q"])
    path8 = (synth.to_e4m3(x["q_idx"]), x["w"], synth.to_e4m3(x["k_idx"]), x["q"])
    tail = (x["gate"], x["q_pos"])
    scores = sga.index_scores(*path[:3], x["q_pos"])  # the queries are the last positions: every entry is written
    idx, out = sga.forward(*path, x["kv"], *tail)
    pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    kv4 = sga.kv4_append(x["kv"], pos, torch.zeros((B, L, sga.KV4_ROW_BYTES), dtype=torch.uint8, device="cuda"))
    codes, scale = sga.quantize_fp8(x["kv"])
    w_scale = scale[0, ::128].contiguous()
    D, R = 512, 144
    h = torch.randn((B, T, D), generator=g, device="cuda").to(torch.bfloat16)

    def weight(rows, cols):
        return torch.randn((rows, cols), generator=g, device="cuda") * cols ** -0.5

    bf = torch.bfloat16
    uk = {n: weight(64 * 128, 512).to(bf).view(64, 128, 512) for n in ("w_uk", "w_uv")}
    wts = dict(uk, w_hq=weight(R + 768, D).to(bf), w_cq=weight(20544, R).to(bf), w_o=weight(D, 8192).to(bf))
    wts8 = dict(uk)
    for n, rows, cols in (("w_hq", 256 + 832, D), ("w_cq", 20608, R), ("w_o", D, 8192)):
        wts8[n] = (weight(rows, cols) * 64).to(torch.float8_e4m3fn)
        wts8[n + "_scale"] = torch.full((-(-rows // 128), -(-cols // 128)), 2.0 ** -6, device="cuda")
    kv, k_idx = x["kv"].clone(), x["k_idx"].clone()
    kv4_l, k_idx8 = kv4.clone(), x["k_idx"].clone()
    return {
        "index_scores": lambda s: sga.index_scores(*path[:3], x["q_pos"], stream=s),
        "index_scores_fp8": lambda s: sga.index_scores_fp8(*path8[:3], x["q_pos"], stream=s),
        "topk_select": lambda s: sga.topk_select(scores, x["q_pos"], stream=s),
        "topk_select_noalloc": lambda s: sga.topk_select_noalloc(scores, x["q_pos"], stream=s),
        "sparse_mla_attend": lambda s: sga.sparse_mla_attend(x["q"], x["kv"], idx, x["gate"], stream=s),
        "forward": lambda s: sga.forward(*path, x["kv"], *tail, stream=s),
        "forward_fp8": lambda s: sga.forward_fp8(*path8, x["kv"], *tail, stream=s),
        "forward_fused": lambda s: sga.forward_fused(*path, x["kv"], *tail, stream=s),
        "forward_fused_fp8": lambda s: sga.forward_fused_fp8(*path8, x["kv"], *tail, stream=s),
        "kv4_append": lambda s: sga.kv4_append(x["kv"], pos, kv4, stream=s),
        "kv4_read": lambda s: sga.kv4_read(kv4, pos, stream=s),
        "sparse_mla_attend_kv4": lambda s: sga.sparse_mla_attend_kv4(x["q"], kv4, idx, x["gate"], stream=s),
        "forward_kv4": lambda s: sga.forward_kv4(*path, kv4, *tail, stream=s),
        "quantize_fp8": lambda s: sga.quantize_fp8(x["kv"], stream=s),
        "gemm_fp8": lambda s: sga.gemm_fp8(codes, scale, codes[0], w_scale, stream=s),
        "layer_project": lambda s: list(sga.layer_project(wts, h, x["q_pos"], kv, k_idx, stream=s).values()),
        "layer_output": lambda s: sga.layer_output(wts, out, stream=s),
        "layer_forward": lambda s: sga.layer_forward(wts, h, x["q_pos"], kv, k_idx, stream=s),
        "layer_forward_fp8kv4": lambda s: sga.layer_forward_fp8kv4(wts8, h, x["q_pos"], kv4_l, k_idx8, stream=s),
        "indexer_warmup": lambda s: list(sga.indexer_warmup(*path, x["kv"], idx, stream=s).values()),
    }


CALLS = ["index_scores", "index_scores_fp8", "topk_select", "topk_select_noalloc", "sparse_mla_attend", "forward",
         "forward_fp8", "forward_fused", "forward_fused_fp8", "kv4_append", "kv4_read", "sparse_mla_attend_kv4",
         "forward_kv4", "quantize_fp8", "gemm_fp8", "layer_project", "layer_output", "layer_forward",
         "layer_forward_fp8kv4", "indexer_warmup"]


@pytest.fixture(scope="module")
def calls():
    made = _calls()
    assert list(made) == CALLS
    torch.cuda.synchronize()
    return made


def _copies(result):
    return [t.clone() for t in (result if isinstance(result, (tuple, list)) else [result])]


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_belongs_to_the_given_stream(calls, name):
    """`stream=` alone, without outputs or a workspace, while the current stream is busy: the call neither waits for the
    current stream (on which the workspace's zeros would otherwise be behind everything queued) nor loses its
    workspace to what the current stream allocates and fills right after."""
    call = calls[name]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = _copies(call(s))
    # the sizes once, so that nothing below has to wait for the device's allocator
    fill = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 64 << 20)]
    del fill
    torch.cuda.synchronize()
    current = torch.cuda.current_stream()
    start = time.perf_counter()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = call(s)
    done = torch.cuda.Event()
    done.record(s)
    fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 64 << 20)]
    done.synchronize()
    if time.perf_counter() - start < 0.1:  # else the host was held up, and the current stream may be done by now
        assert not current.query(), "the call waited for the current stream"
    with torch.cuda.stream(s):
        got = _copies(got)
    torch.cuda.synchronize()
    del fill
    for a, b in zip(got, want):
        if name == "indexer_warmup":  # its sums are atomic, in no fixed order
            assert float((a - b).norm()) <= 1e-3 * float(b.norm())
        else:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_stream_of_another_library(calls):
    """Any object with a cuda_stream names a stream."""
    class Foreign:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    s = torch.cuda.Stream()
    for name in ("forward", "forward_kv4", "gemm_fp8", "quantize_fp8"):
        with torch.cuda.stream(s):
            want = _copies(calls[name](s))
        s.synchronize()
        got = calls[name](Foreign(s))
        s.synchronize()
        for a, b in zip(_copies(got), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
