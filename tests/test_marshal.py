"""The Python entry of the operators around the attention: where its memory
comes from, what it holds while it works, what it raises."""
import ctypes
import os
import shutil
import subprocess
import threading
import time

import pytest
import torch

import attention_forward_14_gb300 as af
from attention_forward_14_gb300 import binding
import ops_ref as R

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def norm_inputs(b=2, h=4, hkv=2, s=33, d=64, seed=1):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((b, h, s, d), generator=g).half().to(DEV)
    k = torch.randn((b, hkv, s, d), generator=g).half().to(DEV)
    w = torch.rand(d, generator=g).half().to(DEV)
    return q, k, w, w


def cache_inputs(b=2, h=4, hkv=2, sq=1, d=64, page=64, pages=4, block=16, seed=2):
    g = torch.Generator().manual_seed(seed)
    kp, ks = R.random_pool(b * pages, page, hkv, d, block, seed)
    vp, vs = R.random_pool(b * pages, page, hkv, d, block, seed + 1)
    table = torch.randperm(b * pages, generator=g).reshape(b, pages).to(torch.int32)
    lens = torch.full((b,), page * pages - 3, dtype=torch.int32)
    q = torch.randn((b, h, sq, d), generator=g).half()
    return [t.to(DEV) for t in (q, kp, vp, ks, vs, lens, table)]


# Every call that allocates, at sizes that differ from one to the next.
CALLS = {
    "norm": lambda stream: af.attn_qk_norm_rope(*norm_inputs(), stream=stream),
    "norm backward": lambda stream: af.attn_qk_norm_rope_bwd(*norm_inputs(seed=3)[:2], *norm_inputs(), stream=stream),
    "attention": lambda stream: af.attn_fwd_kvcache_paged_fp8(*cache_inputs(), stream=stream),
    "attention, many rows": lambda stream: af.attn_fwd_kvcache_paged_fp8(*cache_inputs(sq=40), stream=stream),
}


def _held(handle):
    """Bytes that the allocator has from the driver for one stream, and bytes of them in use."""
    torch.cuda.synchronize()
    segments = [s for s in torch.cuda.memory_snapshot() if s["stream"] == handle and s["device"] == 0]
    return sum(s["total_size"] for s in segments), sum(s["allocated_size"] for s in segments)


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_a_given_stream_is_that_streams(name):
    """Nothing is in flight here: only where the memory comes from is looked
    at.  A block that the current stream has let go of must not serve a launch
    on another one, which does not wait for what the block's last user does."""
    here, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(here):
        wanted = CALLS[name](None)                       # from the pool of `here`, workspace and all
        free = [t for t in wanted if t is not None]
        sizes = [t.numel() * t.element_size() for t in free]
        addresses = {t.data_ptr() for t in free}
        torch.cuda.synchronize()
        del wanted, free
        before = _held(here.cuda_stream)[0]
        out = [t for t in CALLS[name](side) if t is not None]
        torch.cuda.synchronize()
    assert not addresses & {t.data_ptr() for t in out}
    assert _held(here.cuda_stream)[0] == before
    total, used = _held(side.cuda_stream)
    assert used >= sum(sizes) and total >= used


@gpu
def test_calls_in_turn_on_the_current_and_on_a_given_stream():
    """Long calls on the current stream and calls on another stream between
    them, nothing waiting for anything: each has what it has alone."""
    sets = [[*norm_inputs(4, 8, 8, 700 + 100 * i, 128, 10 + i)] for i in range(4)]
    grads = [norm_inputs(4, 8, 8, 700 + 100 * i, 128, 20 + i)[:2] for i in range(4)]
    caches = [cache_inputs(4, 8, 2, 1 + 39 * (i % 2), 128, 64, 16, 16, 30 + i) for i in range(4)]
    side = torch.cuda.Stream()

    def calls(i, stream):
        return (*af.attn_qk_norm_rope(*sets[i], stream=stream), *af.attn_qk_norm_rope_bwd(*grads[i], *sets[i], stream=stream),
                *af.attn_fwd_kvcache_paged_fp8(*caches[i], stream=stream))

    want = []
    for i in range(4):
        want.append([t.clone() for t in calls(i, None)])
        torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = [[], [], [], []]
    for _ in range(6):
        for i in range(4):
            got[i].append(calls(i, side if i % 2 else None))
            if i % 2 == 0:
                calls(i, None)  # its outputs are let go at once
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(a, w) for r in got[i] for a, w in zip(r, want[i]))


@gpu
def test_an_output_on_a_given_stream_outlives_its_use_on_the_current_one():
    """It is let go while the current stream still reads it: its memory is not
    handed out again before that is done."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, k, w, _ = norm_inputs(2, 8, 8, 2000, 128)
    want = af.attn_qk_norm_rope(q, k, w, w)[0]
    torch.cuda.synchronize()
    copies = []
    for _ in range(20):
        o, _ = af.attn_qk_norm_rope(q, k, w, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copies.append(o + 0)
        del o, _
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in copies)


class _StandIn:
    """A library in place of the loaded one, whose functions sleep and succeed."""
    SOURCE = r"""
#include <stdint.h>
#include <unistd.h>
const char *last_error(void) { return ""; }
int slow(void) { usleep(300000); return 0; }
int64_t bytes(void) { return 1 << 20; }
"""

    def __init__(self, folder):
        src, out = os.path.join(folder, "slow.c"), os.path.join(folder, "slow.so")
        with open(src, "w") as f:
            f.write(self.SOURCE)
        subprocess.run(["gcc", "-shared", "-fPIC", "-o", out, src], check=True)
        lib = ctypes.CDLL(out)
        names = {"attn_last_error": "last_error", "attn_qk_norm_rope_bwd_workspace_bytes": "bytes",
                 "attn_fwd_kvcache_paged_fp8_workspace_bytes": "bytes"}
        for n in binding._MARSHALLED:
            setattr(self, n, getattr(lib, names.get(n, "slow")))


@gpu
@pytest.mark.skipif(shutil.which("gcc") is None, reason="builds a small library")
@pytest.mark.parametrize("name", [*CALLS, "append"])
def test_other_threads_run_while_a_call_works(name, tmp_path):
    """Nothing is launched: the library is one whose functions take 0.3 s."""
    binding.load()
    if name == "append":
        q, kp, vp, ks, vs, lens, table = cache_inputs()
        call = lambda: af.attn_kvcache_append_paged(q[:, :2], q[:, :2], kp, vp, lens, table, k_scale=ks, v_scale=vs)  # noqa: E731
    else:
        call = lambda: CALLS[name](None)  # noqa: E731
    saved, beats, stop = binding._lib, [], threading.Event()

    def beat():
        while not stop.wait(0.005):
            beats.append(time.monotonic())

    other = threading.Thread(target=beat)
    binding._lib = _StandIn(str(tmp_path))
    try:
        call()
        other.start()
        begun = time.monotonic()
        call()
        ended = time.monotonic()
    finally:
        stop.set()
        binding._lib = saved
        binding._marshal()
        if other.ident:
            other.join()
    assert ended - begun >= 0.3
    during = sum(begun < t < ended for t in beats)
    assert during >= 10, during


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_running_out_of_memory_raises_what_torch_raises(name):
    """The limit is the allocator's own, for this process.  A call that fails
    so leaves nothing behind, and the same call works afterwards."""
    want = CALLS[name](None)
    torch.cuda.synchronize()
    norm, cache = norm_inputs(4, 16, 16, 2048, 128), cache_inputs(4, 128, 1, 512, 128)
    call = {"norm": lambda: af.attn_qk_norm_rope(*norm),
            "norm backward": lambda: af.attn_qk_norm_rope_bwd(*norm[:2], *norm),
            "attention": lambda: af.attn_fwd_kvcache_paged_fp8(*cache),
            "attention, many rows": lambda: af.attn_fwd_kvcache_paged_fp8(*cache)}[name]
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (4 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    call()
    got = CALLS[name](None)
    torch.cuda.synchronize()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_a_given_stream_within_a_capture():
    """Calls on a stream that the capturing one has forked, whose memory is
    the graph's; eager calls of the same sizes run between the replays."""
    q, k, w, _ = norm_inputs(4, 8, 8, 300, 128, 50)
    cache = cache_inputs(4, 8, 2, 60, 128, 64, 8, 16, 51)
    side = torch.cuda.Stream()

    def step(stream):
        a, b = af.attn_qk_norm_rope(q, k, w, w, stream=stream)
        grads = af.attn_qk_norm_rope_bwd(a, b, q, k, w, w, stream=stream)
        return (a, b, *grads, *af.attn_fwd_kvcache_paged_fp8(*cache, stream=stream))

    want = [t.clone() for t in step(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        step(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_calls_from_several_threads():
    """Each on a stream of its own, and all at once: the lock is let go."""
    sets = [(norm_inputs(3, 8, 8, 200 + 50 * i, 128, 60 + i), cache_inputs(2, 8, 2, 1 + 25 * i, 128, 64, 8, 16, 70 + i))
            for i in range(4)]

    def step(i, stream):
        norm, cache = sets[i]
        a, b = af.attn_qk_norm_rope(*norm, stream=stream)
        return (a, b, *af.attn_qk_norm_rope_bwd(a, b, *norm, stream=stream),
                *af.attn_fwd_kvcache_paged_fp8(*cache, stream=stream))

    want = [[t.clone() for t in step(i, None)] for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    wrong, gate = [], threading.Barrier(4)

    def work(i):
        try:
            gate.wait(10)
            for n in range(30):
                if n % 2:
                    got = step(i, streams[i])
                else:
                    with torch.cuda.stream(streams[i]):
                        got = step(i, None)
                streams[i].synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append((i, n))
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
