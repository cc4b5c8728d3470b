"""GPU: low-rank adapters by row against a plain 64-bit implementation.

Tolerance: A x is a sum in fp32 (2^-18 sum |a x| bounds its error for the lengths here) that enters the second
product as two bf16 halves (2^-16 of it at most), whose sum in fp32 is off by 2^-18 sum |b v|; the addition to Y
rounds once more in fp32, and the result once to bf16 (2^-8 |ref|)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


def normal(seed, *shape, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def rows_apart(x, pad):
    """The same matrix with `pad` values between its rows, which hold NaN."""
    t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    t[:, : x.shape[1]] = x
    return t[:, : x.shape[1]]


def case(T, L, R, K, N, seed, none=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, L, T)
    ids[rng.random(T) < none] = -1
    return dict(X=normal(seed, T, K), Y=normal(seed + 1, T, N), A=normal(seed + 2, L, R, K, scale=K ** -0.5),
                B=normal(seed + 3, L, N, R, scale=R ** -0.5), ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                scales=torch.tensor(rng.uniform(-2, 2, L), dtype=torch.float32, device="cuda"))


def check(c, out, scales=True, ids=None):
    ids = c["ids"] if ids is None else ids
    ref = c["Y"].double()
    tol = torch.zeros_like(ref)
    for a in range(c["A"].shape[0]):
        rows = (ids == a).nonzero().squeeze(1)
        if rows.numel() == 0:
            continue
        A, B, x = c["A"][a].double(), c["B"][a].double(), c["X"][rows].double()
        s = c["scales"][a].double() if scales else 1.0
        v = x @ A.t()
        ref[rows] += s * (v @ B.t())
        tol[rows] = abs(s) * ((2.0 ** -18 * (x.abs() @ A.abs().t()) + 2.0 ** -15 * v.abs()) @ B.abs().t()) + 2.0 ** -22 * ref[rows].abs()
    assert torch.isfinite(out).all()
    err = (out.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + tol).all(), float((err / (ref.abs() + tol)).max())
    plain = (ids < 0).nonzero().squeeze(1)
    assert torch.equal(out[plain], c["Y"][plain])


SIZES = [(1, 1, 8, 8, 8), (1, 3, 16, 7168, 4096), (2, 5, 24, 72, 264), (15, 4, 32, 200, 40), (16, 2, 8, 1544, 512), (17, 300, 16, 320, 248),
         (45, 9, 8, 1544, 2112), (100, 3, 128, 64, 72), (256, 64, 16, 640, 1024), (513, 5, 40, 264, 520), (600, 4, 64, 128, 256),
         (700, 3, 72, 1000, 136), (1500, 2, 128, 512, 264), (3000, 200, 16, 256, 512),
         # both sides of where a row's two products are one launch: the rows, K, R K and R N
         (512, 6, 8, 2048, 1024), (513, 6, 8, 2048, 1024), (9, 3, 16, 2056, 128), (33, 3, 32, 1032, 128), (70, 9, 16, 128, 2056),
         (20, 2, 32, 1024, 1024), (130, 7, 40, 128, 136), (300, 11, 48, 264, 72), (5, 2, 16, 2312, 264),
         (15, 3, 16, 2048, 2448), (15, 3, 16, 2048, 2456), (16, 3, 64, 1024, 536), (16, 3, 64, 1024, 544), (9, 2, 104, 72, 600),
         (77, 2, 120, 40, 776), (3, 1, 8, 4096, 64), (3, 1, 8, 4104, 64), (1024, 5, 40, 264, 136), (1025, 5, 40, 264, 136),
         (1030, 70, 24, 264, 72), (60, 1, 24, 40, 4120), (33, 2, 8, 16, 12000),
         # two launches, few rows a workgroup
         (5, 3, 16, 4168, 264), (33, 20, 24, 4168, 136), (70, 9, 32, 4104, 264), (130, 7, 48, 2400, 264), (300, 11, 72, 1400, 136),
         (256, 64, 16, 7168, 512), (20, 4, 128, 1000, 1000), (40, 13, 104, 1200, 264), (400, 2, 24, 4160, 264), (63, 40, 48, 2104, 264),
         (64, 40, 48, 2104, 264), (256, 3, 128, 400, 776), (257, 3, 128, 400, 776), (200, 12, 72, 2200, 136), (150, 30, 32, 1400, 3600)]


@pytest.mark.parametrize("T,L,R,K,N", SIZES)
def test_against_plain(T, L, R, K, N):
    c = case(T, L, R, K, N, seed=T + R)
    out = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"])
    check(c, out)
    order = c["ids"].argsort(stable=True).int()
    assert torch.equal(fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"], order=order), out)
    place = c["Y"].clone()
    assert fg.lora_add(place, c["X"], c["A"], c["B"], c["ids"], c["scales"], out=place) is place
    assert torch.equal(place, out)
    check(c, fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"]), scales=False)
    assert fg.read_device_error() == 0


@pytest.mark.parametrize("T,L,R,K,N", [(2, 2, 8, 64, 72), (37, 5, 16, 328, 264), (600, 3, 32, 128, 128)])
def test_rows_apart(T, L, R, K, N):
    """Columns of wider matrices: what stands between the rows is neither read into results nor written."""
    c = case(T, L, R, K, N, seed=T)
    want = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"])
    wide = torch.full((T, N + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    got = fg.lora_add(rows_apart(c["Y"], 24), rows_apart(c["X"], 8), c["A"], c["B"], c["ids"], c["scales"], out=wide[:, 8:N + 8])
    assert torch.equal(got, want) and (wide[:, :8] == 5).all() and (wide[:, N + 8:] == 5).all()


@pytest.mark.parametrize("T", [1, 16, 40, 700])
def test_no_adapter_at_all(T):
    c = case(T, 3, 16, 64, 72, seed=1, none=2.0)
    c["Y"][0, :2] = torch.tensor([-0.0, float("nan")])
    out = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"])
    assert torch.equal(out.view(torch.int16), c["Y"].view(torch.int16))


def test_values_that_are_not_finite_stay_with_their_rows():
    """An adapter full of infinities and NaN, and rows of them, change no row of another adapter."""
    c = case(50, 4, 24, 136, 264, seed=9)
    want = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"])
    A, B, X = c["A"].clone(), c["B"].clone(), c["X"].clone()
    A[2], B[2] = float("inf"), float("nan")
    X[c["ids"] < 0] = float("nan")
    X[7], want[7] = float("nan"), float("nan")
    got = fg.lora_add(c["Y"], X, A, B, c["ids"], c["scales"])
    rows = c["ids"] != 2
    rows[7] = False
    assert torch.equal(got[rows], want[rows])
    if c["ids"][7] >= 0:
        assert got[7].isnan().all()
    assert got[c["ids"] == 2].isnan().all()


def test_ids_and_order_out_of_range():
    c = case(40, 4, 16, 64, 72, seed=3)
    ids = c["ids"].clone()
    ids[5], ids[11] = 4, 1 << 30
    fg.read_device_error()
    out = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], ids, c["scales"])
    assert fg.read_device_error() == fg.DEVERR_BAD_INDEX
    ids[5] = ids[11] = -1
    check(c, out, ids=ids)
    order = torch.arange(40, dtype=torch.int32, device="cuda")
    order[3], order[20] = -1, 40
    kept = torch.full_like(c["Y"], 3.0)
    fg.lora_add(c["Y"], c["X"], c["A"], c["B"], ids, c["scales"], order=order, out=kept)
    assert fg.read_device_error() == fg.DEVERR_BAD_INDEX
    named = torch.ones(40, dtype=torch.bool, device="cuda")
    named[3] = named[20] = False
    assert torch.equal(kept[named], out[named]) and (kept[~named] == 3).all()


def test_rows_do_not_depend_on_their_neighbours():
    """A row's result has the same bits whatever other adapters stand beside it (batches of one launch shape)."""
    c = case(64, 8, 16, 256, 264, seed=5, none=0.0)
    out = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"])
    p = torch.randperm(64, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    moved = fg.lora_add(c["Y"][p], c["X"][p], c["A"], c["B"], c["ids"][p])
    assert torch.equal(moved, out[p])
