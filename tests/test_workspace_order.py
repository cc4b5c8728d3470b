"""Calls of several host threads on one stream: the launches of a call that passes results through the
stream's workspace follow each other, with no other user of that workspace between them.

The library's own host code runs here without a GPU, against HIP calls that record the launches
(hip_record.cpp); no kernel runs and no pointer is followed."""
import ctypes
import os
import subprocess
import sys
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 1 << 20


def compiled(tmp_path):
    so = str(tmp_path / "hip_record.so")
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1",
                           "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
                           os.path.join(HERE, "hip_record.cpp"), "-o", so, "-pthread"])
    return so


def in_a_process(tmp_path, name, file=__file__):
    """Run a function of a test file where the recording calls are found before the real ones."""
    lib = os.path.join(os.path.dirname(HERE), "fp8_block_scaled_x128_amd", "libfp8gemm.so")
    if not os.path.exists(lib):
        subprocess.check_call([sys.executable, "-m", "fp8_block_scaled_x128_amd.build"], cwd=os.path.dirname(HERE))
    r = subprocess.run([sys.executable, os.path.abspath(file), name, compiled(tmp_path)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


class Recorded:
    def __init__(self, so):
        self.hip = ctypes.CDLL(so, mode=ctypes.RTLD_GLOBAL)
        sys.path.insert(0, os.path.dirname(HERE))
        import fp8_block_scaled_x128_amd as fg
        assert "torch" not in sys.modules
        self.lib = fg.lib()
        self.hip.record_launches.restype = ctypes.c_int64
        self.hip.record_launches.argtypes = [ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64]

    def launches(self, first=0):
        """(thread, stream, blocks, threads) of every launch from `first` on."""
        n = self.hip.record_launches(first, None, 0) - first
        buf = (ctypes.c_int64 * (4 * n))()
        self.hip.record_launches(first, buf, n)
        return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]

    def dispatch(self, stream, T=2000, k=8, G=16, H=256):
        return self.lib.fp8gemm_moe_dispatch_contiguous(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, T, H, k, G, T * k + 128 * G, 0, stream)

    def dispatch_masked(self, stream, T=1500, k=8, G=32, H=128):
        return self.lib.fp8gemm_moe_dispatch_masked(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, T, H, k, G, 1000, 0, stream)

    def split_k(self, stream):
        return self.lib.fp8gemm_nt(FAKE, FAKE, FAKE, FAKE, FAKE, 64, 2112, 7168, stream)

    def stream_k(self, stream):
        return self.lib.fp8gemm_nt(FAKE, FAKE, FAKE, FAKE, FAKE, 4096, 1536, 7168, stream)


def _threads_on_one_stream(so):
    r = Recorded(so)
    stream, calls = 0x1230, 12
    assert r.dispatch(stream) == 0
    assert len(r.launches()) == 4                    # count, sums, copy, scales
    assert r.split_k(stream) == 0 and r.stream_k(stream) == 0
    assert len(r.launches()) == 6
    start, bad, owner = 6, [], {}

    def work(calls_of, launches):
        owner[threading.get_native_id()] = launches
        for _ in range(calls):
            for f in calls_of:
                if f(stream) != 0:
                    bad.append(f)
    threads = [threading.Thread(target=work, args=a) for a in
               (([r.dispatch], 4), ([r.dispatch_masked], 4), ([r.dispatch], 4), ([r.split_k, r.stream_k], 1))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not bad
    log = r.launches(start)
    assert len(log) == calls * (4 + 4 + 4 + 2)
    at, turns = 0, 0
    while at < len(log):
        tid = log[at][0]
        n = owner[tid]
        assert [x[0] for x in log[at:at + n]] == [tid] * n, "launch %d: another thread's launch within a call" % at
        turns += at > 0 and log[at - 1][0] != tid
        at += n
    assert turns >= 3                                # the threads did take turns


def test_launches_of_a_call_are_not_separated(tmp_path):
    in_a_process(tmp_path, "_threads_on_one_stream")


def _streams_do_not_wait(so):
    """A call on one stream goes on while another stream's is being enqueued."""
    r = Recorded(so)
    r.hip.record_pause(20000)
    assert r.dispatch(0x1230) == 0 and r.dispatch(0x4560) == 0
    start = len(r.launches())
    threads = [threading.Thread(target=r.dispatch, args=(s,)) for s in (0x1230, 0x4560)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    streams = [x[1] for x in r.launches(start)]
    assert sorted(streams) == [0x1230] * 4 + [0x4560] * 4
    assert sum(a != b for a, b in zip(streams, streams[1:])) > 1, streams


def test_streams_do_not_wait_for_each_other(tmp_path):
    in_a_process(tmp_path, "_streams_do_not_wait")


def _per_thread_stream(so):
    """The per-thread default stream is a stream of its own in every host thread, with its own workspace (two
    allocations); other streams' are shared by the threads."""
    r = Recorded(so)
    r.hip.record_pause(0)
    per_thread = 2                                   # hipStreamPerThread
    for stream, workspaces in ((0x1230, 1), (per_thread, 3), (None, 1)):
        before = r.hip.record_allocations()
        for _ in range(2):
            assert r.split_k(stream) == 0 and r.dispatch(stream) == 0
        threads = [threading.Thread(target=lambda: (r.split_k(stream), r.dispatch(stream), r.split_k(stream))) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(120)
        assert r.hip.record_allocations() - before == 2 * workspaces, stream


def test_the_per_thread_stream_has_a_workspace_per_thread(tmp_path):
    in_a_process(tmp_path, "_per_thread_stream")


def _failed_allocation(so):
    """Where a workspace cannot be allocated the call reports it, nothing is kept, and the next calls go on."""
    r = Recorded(so)
    r.hip.record_pause(0)
    for first in (0, 1):                             # the partials' allocation fails; the counters' does
        stream = 0x1000 + first
        r.hip.record_fail_after(first)
        before, frees, n = r.hip.record_allocations(), r.hip.record_frees(), len(r.launches())
        assert r.split_k(stream) == 6                # FP8GEMM_ERR_HIP
        assert len(r.launches()) == n and r.hip.record_allocations() - before == r.hip.record_frees() - frees == first
        r.hip.record_fail_after(-1)
        route = r.lib.fp8gemm_route_topk(FAKE, None, FAKE, FAKE, 4, 64, 2, 0, 0, 1, 1, 1, 1, 1.0, stream)
        assert route == 0                            # the failure before is not its own
        assert r.dispatch(stream) == 0 and r.split_k(stream) == 0
        assert r.hip.record_allocations() - before == first + 2


def test_a_failed_allocation_leaves_nothing(tmp_path):
    in_a_process(tmp_path, "_failed_allocation")


if __name__ == "__main__":
    globals()[sys.argv[1]](sys.argv[2])
