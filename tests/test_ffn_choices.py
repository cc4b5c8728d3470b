"""What the launch shapes of the gated block, its gradients and the adapters are chosen by: the host code, run against recorded
HIP calls.  CPU only."""
import ctypes
import os
import random
import re
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from test_workspace_order import FAKE, Recorded, in_a_process  # noqa: E402


class Choices(Recorded):
    def __init__(self, so):
        super().__init__(so)
        self.hip.record_pause(0)

    def config(self):
        buf = ctypes.create_string_buffer(512)
        assert self.lib.fp8gemm_last_config(buf, 512) == 0
        return buf.value.decode()

    def gated(self, M, I, K, at=0, pre=None):
        assert self.lib.fp8gemm_gated_ffn(FAKE + at, FAKE, FAKE, pre, M, I, K, 0, 0x10) == 0
        return self.config()

    def lora(self, T, R, K, N, L=64):
        assert self.lib.fp8gemm_lora_add(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, T, L, R, K, N, K, N, N, 0x10) == 0
        return self.config()

    def backward(self, M, I, K, at=0, pre=None, dX=FAKE, dW=FAKE):
        assert self.lib.fp8gemm_gated_ffn_backward(FAKE, FAKE + at, FAKE, pre, FAKE + at, dX, dW, M, I, K, 0, 0x10) == 0
        return self.config()


def chosen(config):
    """The tiles and K splits in a configuration's words."""
    return re.findall(r"tile=\S+ split=\d+|\brows\b|together=\d", config)


def _addresses(so):
    r = Choices(so)
    rng = random.Random(1)
    for _ in range(300):
        M, I, K = (int(2 ** rng.uniform(*e)) for e in ((0, 12), (3, 8), (3, 10)))
        size = (M, 8 * I, 8 * K)
        for at in (16, 64, 112):
            assert chosen(r.gated(*size, at=at)) == chosen(r.gated(*size)) != [], (size, at)
            assert chosen(r.backward(*size, at=at)) == chosen(r.backward(*size)) != [], (size, at)


def test_addresses_choose_nothing(tmp_path):
    """Sizes alone choose tiles and K splits, and with them the order of the sums: the same matrices anywhere in memory
    give the same bits."""
    in_a_process(tmp_path, "_addresses", __file__)


TILES = {"256x256": 2, "128x256": 3, "128x128": 4, "64x64": 4, "64x64x2": 2}       # and slices of their rings


def _words(so):
    r = Choices(so)
    M, I, K = 333, 264, 712
    for name, ring in TILES.items():
        bm, bn = (int(n) for n in name.split("x")[:2])
        tile = "tile=%dx%dx%d" % (bm, bn, ring)
        for split in (1, 2, 3):
            os.environ["FP8GEMM_FORCE_CONFIG"] = "product:%s:%d" % (name, split)

            def units(rows, cols):
                return -(-rows // bm) * -(-cols // bn) * split
            for dX, dW in ((FAKE, FAKE), (FAKE, None), (None, FAKE)):
                n = len(r.launches())
                words = r.backward(M, I, K, pre=FAKE, dX=dX, dW=dW)
                there, none = "%s split=%d" % (tile, split), "tile=0x0x0 split=0"
                lines = " lines=%d" % (dX is not None and ring == 4)                  # (rows of dpre start beside the lines)
                assert " kept together=%d " % (dX is not None and dW is not None) in words, words
                assert "dX %s%s " % (there if dX else none, lines) in words and words.endswith("dW " + (there if dW else none)), words
                assert sum(x[2] for x in r.launches(n)[1:]) == (units(M, K) if dX else 0) + (units(2 * I, K) if dW else 0)
            n = len(r.launches())
            words = r.backward(M, I, K)
            assert words.endswith("dW %s split=%d products %s split=%d lines=0" % (tile, split, tile, split)) or name == "64x64x2", words
            got = r.launches(n)
            assert got[0][2] == -(-M // bm) * -(-2 * I // bn) * split or name == "64x64x2"     # (a shape of the gradients)
    del os.environ["FP8GEMM_FORCE_CONFIG"]
    assert " rows together=" in r.backward(3, 2048, 7168) and r.gated(3, 2048, 7168).endswith(" rows")


def test_words_name_the_tiles_that_are_launched(tmp_path):
    in_a_process(tmp_path, "_words", __file__)


PER_CU = {"256x256": 1, "128x256": 1, "128x128": 1, "64x64": 2}                    # workgroups of a tile that share a CU


def _cap(so):
    r = Choices(so)
    rng = random.Random(2)
    sizes = [(64, 2048, 7168), (300, 512, 7168)] + [tuple(int(2 ** rng.uniform(*e)) * m for e, m in (((5, 11), 1), ((3, 8), 8), ((3, 10), 8)))
                                                    for _ in range(100)]
    adapters = [(16, 16, 7168, 4096), (256, 16, 7168, 4096), (2000, 128, 7168, 4096), (8192, 32, 7168, 4096)]
    free = [r.gated(*s) for s in sizes] + [r.backward(*s) for s in sizes] + [r.lora(*s) for s in adapters]
    fewer = 0
    for cap in (1, 7, 24, 100):
        assert r.lib.fp8gemm_set_num_cus(cap) == 0
        for i, s in enumerate(sizes):
            n = len(r.launches())
            words = r.gated(*s)
            tile, split = re.search(r"tile=(\S+) split=(\d+)", words).groups()
            assert split == "1" or r.launches(n)[0][2] <= cap * PER_CU[tile], (cap, words)
            fewer += words != free[i]
            r.backward(*s)
        for T, R, K, N in adapters:
            n = len(r.launches())
            words = r.lora(T, R, K, N)
            rows, split = (int(x) for x in re.search(r"rows=(\d+) split=(\d+)", words).groups())
            tiles = -(-T // rows)
            assert split == 1 or tiles * split <= 2 * cap, (cap, words)
            assert [x[2] for x in r.launches(n)][0] == tiles * split * (-(-R // 32) if rows < 64 else 2)
        n = len(r.launches())
        r.lora(140000, 128, 64, 64, L=3)                       # the workspace, and with it the passes, stay as they are
        assert len(r.launches()) - n == 4
    assert fewer > 50
    assert r.lib.fp8gemm_set_num_cus(0) == 0
    assert free == [r.gated(*s) for s in sizes] + [r.backward(*s) for s in sizes] + [r.lora(*s) for s in adapters]


def test_launch_shapes_go_by_the_cap(tmp_path):
    in_a_process(tmp_path, "_cap", __file__)


if __name__ == "__main__":
    globals()[sys.argv[1]](sys.argv[2])
