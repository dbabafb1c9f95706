"""The layer norm, the dropout and the gated projection past 2^32 elements (GPU).
The last rows of a large call are compared with a small call on those rows, or
with the formula in 64 bits."""

import pytest
import torch

import ln64
import swiglu_backward_int8_amd as sq
from test_operator_limits_gpu import filled, new

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
bf16, f32 = torch.bfloat16, torch.float32
RNG = (77, 5)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sq.lib()
    yield
    torch.cuda.empty_cache()


def rng():
    return torch.tensor(RNG, dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("D,group", [(4096, 128), (1000, 64)])
def test_norm(D, group):
    T = 2**32 // D + 77
    x = filled(T, D)
    w = (1 + 0.1 * torch.randn(D, device=DEV)).bfloat16()
    b = (0.1 * torch.randn(D, device=DEV)).bfloat16()

    def forward(x):
        T = x.shape[0]
        out = new(T, D, dtype=torch.int8), new(T, -(-D // group), dtype=f32), new(T, dtype=f32), new(T, dtype=f32)
        sq.layer_norm_quant(x, w, b, out[0], out[1], mean=out[2], rstd=out[3], group_size=group)
        return out

    tail = slice(T - 200, T)
    out = forward(x)
    small = forward(x[tail].clone())
    for a, c in zip(out, small):
        assert torch.equal(a[tail], c)
    # backward: rows are independent; the sums of dy that is zero but in the last rows are theirs alone
    dy = torch.zeros_like(x)
    dy[tail] = filled(200, D, 1)
    dx, dw, db = new(T, D), new(D, dtype=f32), new(D, dtype=f32)
    sq.layer_norm_bwd(dy, x, w, out[2], out[3], dx, dw=dw, db=db, workspace=sq.layer_norm_bwd_workspace(T, D, DEV))
    dxs = new(200, D)
    sq.layer_norm_bwd(dy[tail].clone(), x[tail].clone(), w, small[2], small[3], dxs)
    assert torch.equal(dx[tail], dxs)
    _, _, dw64, dw_size, db64, db_size = ln64.norm_bwd(dy[tail].cpu(), x[tail].cpu(), w.cpu(), small[2].cpu(), small[3].cpu())
    assert ((dw.cpu().double() - dw64).abs() <= 234 * 2.0**-24 * dw_size + 1e-40).all()
    assert ((db.cpu().double() - db64).abs() <= 232 * 2.0**-24 * db_size + 1e-40).all()


@pytest.mark.parametrize("D", [4096, 1001])
def test_dropout(D):
    T = 2**32 // D + 77
    x = torch.ones((T, D), dtype=bf16, device=DEV)
    sq.dropout_add(x, x, 0.25, rng())
    # the mask of the last rows, from the oracle's words at those rows
    rows = 60
    want = kept_rows(T - rows, rows, D, 0.25)
    assert torch.equal((x[T - rows:] != 0).cpu(), want)
    assert torch.equal((x[:rows] != 0).cpu(), ln64.kept(RNG, rows, D, 0.25))


def kept_rows(first, rows, D, p):
    """ln64.kept of rows first and on: the row is the counter's second word."""
    seed, step = RNG
    out = torch.empty((rows, D), dtype=torch.bool)
    for i in range(rows):
        for block in range(-(-D // 4)):
            c, k = [block, first + i, step % 2**32, step >> 32], [seed % 2**32, seed >> 32]
            for _ in range(10):
                a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
                c = [(b >> 32) ^ c[1] ^ k[0], b % 2**32, (a >> 32) ^ c[3] ^ k[1], a % 2**32]
                k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
            for j in range(min(4, D - 4 * block)):
                out[i, 4 * block + j] = c[j] >= round(p * 2**32)
    return out


@pytest.mark.parametrize("T,H,D", [(200000, 11008, 64), (2**20 + 40, 4104, 8), (70000, 40, 65536)])
def test_projection(T, H, D):
    # small whole numbers: sums that fp32 holds exactly
    g = torch.Generator(device=DEV).manual_seed(1)
    x = new(T, D)
    for i in range(0, T, 4099):  # a few thousand random rows, repeated
        n = min(4099, T - i)
        x[i:i + n] = torch.randint(-2, 3, (n, D), generator=g, device=DEV).to(bf16)
    w = torch.randint(-2, 3, (2 * H, D), generator=g, device=DEV).to(bf16)
    gu, y = new(T, 2 * H), new(T, H)
    sq.swiglu_gemm(x, w, y, gu=gu)
    tail = slice(T - 60, T)
    want = x[tail].double() @ w.double().t()
    assert torch.equal(gu[tail], want.to(bf16))
    small = new(60, H)
    sq.swiglu_gemm(x[tail].clone(), w, small)
    assert torch.equal(y[tail], small)  # exact sums, the same formula
    # backward: dy is zero but in the last rows, gates 0 or 64 there
    dy, d_gu = torch.zeros_like(y), new(T, 2 * H)
    dy[tail] = torch.randint(-2, 3, (60, H), generator=g, device=DEV).to(bf16)
    gu[tail, :H] = 64 * torch.randint(0, 2, (60, H), generator=g, device=DEV).to(bf16)
    gu[tail, H:] = torch.randint(-1, 2, (60, H), generator=g, device=DEV).to(bf16)
    dx, dw = new(T, D, dtype=f32), new(2 * H, D, dtype=f32)
    ws = sq.swiglu_gemm_bwd_workspace(T, H, D, DEV)
    sq.swiglu_gemm_bwd(dy, gu, x, w, d_gu, dx=dx, dw=dw, workspace=ws)
    gate, up, d = gu[tail, :H].double(), gu[tail, H:].double(), dy[tail].double()
    d = torch.cat([d * up * torch.where(gate == 0, 0.5, 1.0), d * gate], 1)
    assert torch.equal(d_gu[tail].double(), d)
    assert torch.equal(dx[tail].double(), d @ w.double())
    assert bool((dx[:T - 60] == 0).all())
    assert torch.equal(dw.double(), d.t() @ x[tail].double())


@pytest.mark.parametrize("T,H,D", [(8, 16, 2**20), (300, 8, 2**20), (8, 2**20, 8), (40, 2**20, 16), (2**22, 8, 8)])
def test_projection_at_the_ends_of_the_sizes(T, H, D):
    g = torch.Generator(device=DEV).manual_seed(2)
    pick = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV).to(bf16)
    x, w, dy = pick(T, D), pick(2 * H, D), pick(T, H)
    y, gu = new(T, H), new(T, 2 * H)
    sq.swiglu_gemm(x, w, y, gu=gu)
    rows = slice(max(0, T - 100), T)
    assert torch.equal(gu[rows], (x[rows].double() @ w.double().t()).to(bf16))
    gu[:, :H] = 0
    gu[:, H:] = pick(T, H)
    dx, dw = new(T, D, dtype=f32), new(2 * H, D, dtype=f32)
    sq.swiglu_gemm_bwd(dy, gu, x, w, gu, dx=dx, dw=dw, workspace=sq.swiglu_gemm_bwd_workspace(T, H, D, DEV))
    assert torch.equal(dx[rows].double(), gu[rows].double() @ w.double())
    columns = slice(max(0, D - 4096), D)
    assert torch.equal(dw[:, columns].double(), gu.double().t() @ x[:, columns].double())
