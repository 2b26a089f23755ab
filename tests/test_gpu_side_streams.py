"""Calls on a stream that is not the current one, on two streams at once, and
beside other Python threads."""
import ctypes
import threading
import time

import pytest
import torch

from test_gpu_fp4 import case
from top_sparse_attention_qsa_b200 import workloads as W

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"


@pytest.fixture(scope="module")
def C():
    from top_sparse_attention_qsa_b200 import _capi
    return _capi


def calls(C):
    """Every call that makes its own outputs, as f(stream) -> tuple of tensors."""
    T, S, heads, K = 40, 8000, (24, 2), 650
    q, cache, ks, vs, g = case(C, T, S, heads, seed=95)
    idx = W.random_lists(T, 2, K, S, g, DEV)
    blocks = W.random_lists(T, 2, 64, S // 4, g, DEV)
    k, v = (torch.randn((T, 2, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = C.rope_table(S, 64, device=DEV)
    kc, vc = (torch.randn((S, 2, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    k8, v8 = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    spare = [x.clone() for x in (kc, vc, k8, v8, cache.buffer)]
    qi = torch.randn((T, 4, 128), generator=g, device=DEV).to(torch.bfloat16)
    ki = torch.randn((S // 4, 128), generator=g, device=DEV).to(torch.bfloat16)
    last, first = torch.full((T,), S - 1, dtype=torch.int32, device=DEV), torch.zeros((T,), dtype=torch.int32, device=DEV)
    scores = C.indexer_scores(qi, ki, last, first)
    torch.cuda.synchronize()
    return {
        "kv_append": lambda s: (C.kv_append(k, v, pos, pos, table, spare[0], spare[1], q=q, stream=s),),
        "kv_append_fp8": lambda s: C.kv_append_fp8(k, v, pos, pos, table, spare[2], spare[3], 0.02, 0.02, q=q,
                                                   want_seen=True, stream=s),
        "kv_append_fp4": lambda s: C.kv_append_fp4(k, v, pos, pos, table, C.Fp4Cache(spare[4]), ks, vs, q=q,
                                                   want_seen=True, stream=s),
        "prefill_fp4": lambda s: C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, stream=s),
        "decode_fp4": lambda s: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, stream=s),
        "decode_fp4 workspace": lambda s: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, num_splits=3, stream=s),
        "prefill": lambda s: C.sparse_prefill_fwd(q, kc, vc, idx, stream=s),
        "debug_gather": lambda s: C.sparse_prefill_debug_gather(q, kc, vc, idx, stream=s),
        "block": lambda s: C.sparse_prefill_block_fwd(q, kc, vc, blocks, 4, stream=s),
        "prefill_fp8": lambda s: C.sparse_prefill_fp8_fwd(q, k8, v8, idx, stream=s),
        "debug_gather_lists": lambda s: C.sparse_prefill_debug_gather_lists(q, kc, vc, blocks, 4, stream=s),
        "decode": lambda s: C.sparse_decode_fwd(q, kc, vc, idx, num_splits=3, stream=s),
        "decode_fp8": lambda s: C.sparse_decode_fp8_fwd(q, k8, v8, idx, num_splits=3, stream=s),
        "fold_heads": lambda s: (C.indexer_fold_heads(qi, ki, stream=s),),
        "scores": lambda s: (C.indexer_scores(qi, ki, last, first, stream=s),),
        "scores unfolded": lambda s: (C.indexer_scores(qi, ki, last, first, fold=False, stream=s),),
        "topk": lambda s: C.topk_select(scores, last, first, S // 4, 64, copies=2, stream=s),
        "select": lambda s: C.indexer_select(qi, ki, last, first, 64, stream=s),
    }


NEW = ("kv_append", "kv_append_fp8", "kv_append_fp4", "prefill_fp4", "decode_fp4", "decode_fp4 workspace")


def outputs_belong_to_the_launching_stream(run):
    """Outputs made for a call on another stream are that stream's: once dropped,
    their memory is not given to work of the current stream."""
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del want
    spans = [(x.data_ptr(), x.data_ptr() + x.untyped_storage().nbytes()) for x in got]
    sizes = [x.untyped_storage().nbytes() for x in got]
    del got, a, b
    later = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    for x in later:
        for lo, hi in spans:
            assert x.data_ptr() + x.numel() <= lo or x.data_ptr() >= hi


def test_outputs_of_cache_and_4bit_calls(C):
    every = calls(C)
    for name in NEW:
        outputs_belong_to_the_launching_stream(every[name])


def test_outputs_of_the_other_calls(C):
    every = calls(C)
    for name in every:
        if name not in NEW:
            outputs_belong_to_the_launching_stream(every[name])


def test_forms_of_a_stream_handle(C):
    """The default stream's handle 0, a stream object and a ctypes pointer name a stream as an int does."""
    every = calls(C)
    side = torch.cuda.Stream()
    for name in ("decode", "scores"):
        want = every[name](None)
        torch.cuda.synchronize()
        for s in (0, side, ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p(0)):
            got = every[name](s)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("call", ["append", "prefill", "decode"])
def test_other_threads_run_while_a_launch_waits(C, call):
    """A launch that waits for room in its stream's queue keeps only its own thread waiting."""
    T, S = 2, 64
    q, cache, ks, vs, g = case(C, T, S, (3, 1), seed=96)
    idx = W.random_lists(T, 1, 8, S, g, DEV)
    k = torch.zeros((T, 1, 256), dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = C.rope_table(S, 64, device=DEV)
    out = torch.empty_like(q)
    run = {"append": lambda: C.kv_append_fp4(k, k, pos, pos, table, cache, ks, vs),
           "prefill": lambda: C.sparse_prefill_fp4_fwd(q, cache, idx, ks, vs, out=out, want_lse=False),
           "decode": lambda: C.sparse_decode_fp4_fwd(q, cache, idx, ks, vs, out=out, want_lse=False)}[call]
    run()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    other = threading.Thread(target=tick)
    other.start()
    torch.cuda._sleep(2_000_000_000)                     # about a second of the stream
    begin, longest = time.perf_counter(), (0.0, 0.0, 0.0)
    while time.perf_counter() - begin < 3 and longest[0] < 0.2:
        a = time.perf_counter()
        run()
        b = time.perf_counter()
        longest = max(longest, (b - a, a, b))
    stop.set()
    other.join()
    torch.cuda.synchronize()
    waited, a, b = longest
    assert waited >= 0.2, "the queue never filled"
    during = [t for t in ticks if a <= t <= b]
    assert len(during) > 0.1 * waited / 0.002, f"{len(during)} ticks in {waited:.2f} s"


@pytest.mark.parametrize("heads", [(24, 2), (16, 2)])
def test_two_decodes_through_workspaces_at_once(C, heads):
    """Decodes whose chunks go through a workspace, on two streams at once, as when each runs alone."""
    T, ctx, K, splits = 40, 700, 650, 3
    runs = []
    for seed in (97, 98):
        q, cache, ks, vs, g = case(C, T, T * ctx, heads, seed)
        idx = W.random_lists(T, 2, K, ctx, g, DEV) + (torch.arange(T, dtype=torch.int32, device=DEV) * ctx).view(T, 1, 1)
        assert C.decode_fp4_workspace_bytes(q, cache, idx, splits) > 0
        runs.append((q, cache, idx, ks, vs))
    call = lambda r: C.sparse_decode_fp4_fwd(*r, num_splits=splits)  # noqa: E731
    alone = [call(r) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    outs = []
    for _ in range(20):                                  # workspaces are let go and taken again with kernels in flight
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                outs.append(call(r))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(outs):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(l, alone[i % 2][1])
