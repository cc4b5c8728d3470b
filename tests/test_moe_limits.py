"""The largest sizes of routing, dispatch and combine: a call whose launch would have 2^32 threads or more, or
whose counts do not fit the stream's workspace, is refused on the host, and the last size below is not.
CPU only: the library's host code runs against HIP calls that record the launches (hip_record.cpp)."""
import sys

import test_workspace_order as recorded

FAKE = recorded.FAKE
UNSUPPORTED = 4


def _limits(so):
    r = recorded.Recorded(so)
    r.hip.record_pause(0)
    lib, stream = r.lib, 0x1230

    def route(T):
        return lib.fp8gemm_route_topk(FAKE, None, FAKE, FAKE, T, 1, 1, 1, 0, 1, 1, 1, 1, 1.0, stream)

    def route_wide(T):
        return lib.fp8gemm_route_topk(FAKE, None, FAKE, FAKE, T, 1000, 1, 1, 0, 1, 1, 1, 1, 1.0, stream)

    def route_backward(T):
        return lib.fp8gemm_route_topk_backward(FAKE, FAKE, FAKE, FAKE, T, 1, 1, 1, 0, 1, 1.0, stream)

    def combine(T, H=8):
        return lib.fp8gemm_moe_combine(FAKE, None, FAKE, FAKE, T, H, 1, 1, stream)

    def combine_backward(T, H=8):
        return lib.fp8gemm_moe_combine_backward(FAKE, FAKE, None, FAKE, FAKE, FAKE, T, H, 1, 1, stream)

    def dispatch(T, H=128, G=4):
        return lib.fp8gemm_moe_dispatch_masked(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, T, H, 1, G, 128, 0, stream)

    top = 1 << 28
    for call, last in ((route, top - 17), (route_wide, top - 17), (route_backward, top - 17),
                       (combine, (1 << 24) - 1), (lambda T: combine(T, 2056), (1 << 23) - 1), (combine_backward, (1 << 24) - 1),
                       (lambda T: combine_backward(T, 2056), (1 << 24) - 1),
                       (lambda T: dispatch(T, 1 << 24), 2047), (lambda T: dispatch(T, 16384), (1 << 22) - 1),
                       # words of the workspace: pairs, chunks of 1024 for each expert, two per expert
                       (lambda T: dispatch(T, 128, 1), (1 << 25) * 1024 // 1025 - 2), (lambda T: dispatch(T, 128, 1024), (1 << 24) - 1024)):
        n = len(r.launches())
        assert call(last + 1) == UNSUPPORTED, (call, last)
        assert len(r.launches()) == n                # nothing was enqueued
        assert call(last) == 0, (call, last)
        new = r.launches(n)
        assert new and all(blocks * threads < 1 << 32 for _, _, blocks, threads in new), new


def test_limits(tmp_path):
    recorded.in_a_process(tmp_path, "_limits", __file__)


if __name__ == "__main__":
    globals()[sys.argv[1]](sys.argv[2])
