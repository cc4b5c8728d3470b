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
                assert " kept together=%d " % (dX is not None and dW is not None) in words, words
                assert "dX %s " % (there if dX else none) in words and words.endswith("dW " + (there if dW else none)), words
                assert sum(x[2] for x in r.launches(n)[1:]) == (units(M, K) if dX else 0) + (units(2 * I, K) if dW else 0)
            n = len(r.launches())
            words = r.backward(M, I, K)
            assert words.endswith("dW %s split=%d products %s split=%d" % (tile, split, tile, split)) or name == "64x64x2", words
            got = r.launches(n)
            assert got[0][2] == -(-M // bm) * -(-2 * I // bn) * split or name == "64x64x2"     # (a shape of the gradients)
    del os.environ["FP8GEMM_FORCE_CONFIG"]
    assert " rows together=" in r.backward(3, 2048, 7168) and r.gated(3, 2048, 7168).endswith(" rows")


def test_words_name_the_tiles_that_are_launched(tmp_path):
    in_a_process(tmp_path, "_words", __file__)


if __name__ == "__main__":
    globals()[sys.argv[1]](sys.argv[2])
