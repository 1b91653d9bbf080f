"""The per-worker training operators (embedding, layer norm, distillation)
against their definitions in 64 bits, their refusals, and a run of them
together with the optimizer step.

Bounds.  u = 2^-24 is the most an fp32 rounding is off, relative to the value;
`half` is the same for an output's type (fp32 2^-24, bf16 2^-8).  A sum of n
terms taken one after another in fp32 is off by at most n u times the sum of
the terms' magnitudes.
"""
import itertools
import math

import pytest
import torch

from sign_muon_optimizer_momentum_b200 import _lib as L
from sign_muon_optimizer_momentum_b200 import layers
from sign_muon_optimizer_momentum_b200.step import SignMuonStep

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def half(dtype):
    return torch.finfo(dtype).eps / 2


def even(rows, n):
    return [rows * i // n for i in range(n + 1)]


# ------------------------------------------------------------- CPU: refusals
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        from sign_muon_optimizer_momentum_b200 import build
        build.build()
    return L.load()


def _err(fn, *args):
    with pytest.raises(L.SignMuonError) as e:
        fn(*args)
    return e.value.status


P, ODD = 1 << 20, (1 << 20) + 1   # addresses that are never dereferenced


def test_embedding_refusals(lib):
    def fwd(shape=(10, 8), dt=0, table=P, ld=8, n=4, ids=P, ydt=0, y=P, ldy=8):
        return _err(L.signmuon_embedding_forward, shape, dt, table, ld, n, 1, ids, 1.0, ydt, y, ldy)
    assert fwd(shape=(0, 8)) == 1 and fwd(shape=(10, 0)) == 1 and fwd(shape=(10, -1)) == 1
    assert fwd(dt=2) == 1 and fwd(ydt=7) == 1 and fwd(table=0) == 1 and fwd(ids=0) == 1 and fwd(y=0) == 1
    assert fwd(ld=7) == 1 and fwd(ldy=7) == 1 and fwd(n=-1) == 1
    assert fwd(table=ODD) == 2 and fwd(y=ODD) == 2 and fwd(ids=P + 4) == 2
    assert fwd(shape=(10, (1 << 20) + 1), ld=1 << 21, ldy=1 << 21) == 3
    L.signmuon_embedding_forward((10, 8), 0, P, 8, 0, 1, 0, 1.0, 0, 0, 8)      # no tokens: nothing to do

    def bwd(shape=(10, 8), rows=(0, 2, 4), ids=P, ddt=0, dy=P, ld=8, gdt=0, grad=(P, P), ws=P, nbytes=1 << 20):
        return _err(L.signmuon_embedding_backward, shape, list(rows), 1, ids, ddt, dy, ld, 1.0, 0, gdt, list(grad), ws, nbytes)
    assert bwd(shape=(0, 8)) == 1 and bwd(rows=(0, 3, 2)) == 1 and bwd(rows=(1, 2, 4)) == 1 and bwd(rows=(0,)) == 1
    assert bwd(rows=[0] * 129, grad=[P] * 128) == 1
    assert bwd(ids=0) == 1 and bwd(dy=0) == 1 and bwd(ld=7) == 1 and bwd(grad=(P, 0)) == 1
    assert bwd(ddt=2) == 1 and bwd(gdt=2) == 1
    assert bwd(ids=P + 4) == 2 and bwd(dy=ODD) == 2 and bwd(grad=(P, ODD)) == 2 and bwd(ws=P + 16) == 2
    assert bwd(ws=0) == 4 and bwd(nbytes=512) == 4
    assert bwd(rows=(0, 2, (1 << 30) + 1)) == 3
    size = L.signmuon_embedding_backward_workspace_bytes
    assert size((10, 8), [0, 3, 2]) == 0 and size((0, 8), [0, 3]) == 0 and size((10, 8), [0, 0]) >= 256
    assert size((10, 8), [0, 40]) >= 256 + 4 * 4 * 40 + 2 * 2 * 8 * 4


def test_layer_norm_refusals(lib):
    def fwd(rows=4, cols=8, dt=0, x=P, ld=8, wdt=0, w=P, b=None, eps=1e-5, y=P, ldy=8, mean=P, rstd=P):
        return _err(L.signmuon_layer_norm_forward, rows, cols, dt, x, ld, wdt, w, b, eps, y, ldy, mean, rstd)
    assert fwd(rows=-1) == 1 and fwd(cols=0) == 1 and fwd(dt=3) == 1 and fwd(wdt=3) == 1 and fwd(x=0) == 1 and fwd(y=0) == 1
    assert fwd(w=0) == 1 and fwd(ld=7) == 1 and fwd(ldy=7) == 1 and fwd(mean=0) == 1 and fwd(rstd=0) == 1
    assert fwd(eps=-1.0) == 1 and fwd(eps=math.nan) == 1
    assert fwd(x=ODD) == 2 and fwd(y=ODD) == 2 and fwd(w=ODD) == 2 and fwd(b=ODD) == 2 and fwd(mean=P + 2) == 2
    assert fwd(cols=(1 << 20) + 1, ld=1 << 21, ldy=1 << 21) == 3
    L.signmuon_layer_norm_forward(0, 8, 0, 0, 8, 0, P, None, 1e-5, 0, 8, 0, 0)

    def bwd(cols=8, rows=(0, 4), dt=0, dy=P, ld_dy=8, x=P, ld_x=8, wdt=0, w=P, mean=P, rstd=P, dx=P, ld_dx=8, dw=(P,), db=None,
            ws=P, nbytes=1 << 30):
        return _err(L.signmuon_layer_norm_backward, cols, list(rows), dt, dy, ld_dy, x, ld_x, wdt, w, mean, rstd, dx, ld_dx,
                    list(dw), db, ws, nbytes)
    assert bwd(cols=0) == 1 and bwd(rows=(0, 4, 3), dw=(P, P)) == 1 and bwd(rows=(2, 4)) == 1 and bwd(dt=2) == 1
    assert bwd(dy=0) == 1 and bwd(x=0) == 1 and bwd(dx=0) == 1 and bwd(w=0) == 1 and bwd(mean=0) == 1 and bwd(dw=(0,)) == 1
    assert bwd(db=[0]) == 1 and bwd(ld_dy=7) == 1 and bwd(ld_x=7) == 1 and bwd(ld_dx=7) == 1
    assert bwd(dw=(ODD,)) == 2 and bwd(db=[ODD]) == 2 and bwd(dx=ODD) == 2 and bwd(ws=P + 16) == 2
    assert bwd(ws=0) == 4 and bwd(nbytes=256) == 4
    assert bwd(cols=(1 << 20) + 1, ld_dy=1 << 21, ld_x=1 << 21, ld_dx=1 << 21) == 3
    assert L.signmuon_layer_norm_backward_workspace_bytes(0, [0, 4]) == 0
    assert L.signmuon_layer_norm_backward_workspace_bytes(8, [0, 4, 2]) == 0


def test_distill_refusals(lib):
    def f(vocab=8, rows=(0, 4), dt=0, z=P, ld=8, top=2, ids=P, tdt=0, tl=P, temp=1.0, loss=P, row=P, dz=P, ldd=8, ws=P,
          nbytes=1 << 20):
        return _err(L.signmuon_distill_loss, vocab, list(rows), dt, z, ld, top, 1, ids, tdt, tl, temp, 1.0, loss, row, dz, ldd,
                    ws, nbytes)
    assert f(vocab=0) == 1 and f(rows=(0, 4, 2)) == 1 and f(dt=2) == 1 and f(tdt=2) == 1 and f(z=0) == 1 and f(ld=7) == 1
    assert f(top=0) == 1 and f(top=1025) == 1 and f(ids=0) == 1 and f(tl=0) == 1 and f(loss=0) == 1 and f(row=0) == 1
    assert f(ldd=7) == 1
    for t in (0.0, -1.0, math.inf, math.nan, 1e-7, 1e7):
        assert f(temp=t) == 1
    assert f(vocab=(1 << 30) + 1, ld=1 << 31, ldd=1 << 31) == 3 and f(rows=(0, (1 << 30) + 1)) == 3
    assert f(z=ODD) == 2 and f(dz=ODD) == 2 and f(ids=P + 4) == 2 and f(tl=ODD) == 2 and f(loss=P + 2) == 2 and f(ws=P + 16) == 2
    assert f(ws=0) == 4 and f(nbytes=300) == 4
    assert L.signmuon_distill_workspace_bytes(4, 0) == 0 and L.signmuon_distill_workspace_bytes(-1, 2) == 0


def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: layers.embedding_forward(x, ids), lambda: layers.embedding_backward(ids, x, 8),
                 lambda: layers.layer_norm_forward(x, x[0]), lambda: layers.layer_norm_backward(x, x, x[0], x[:, 0], x[:, 0]),
                 lambda: layers.distill_loss(x, ids.view(4, 1), x[:, :1]),
                 lambda: layers.distill_loss_and_grad(x, ids.view(4, 1), x[:, :1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_shares(lib):
    shares = layers._load().shares
    assert shares(8, 4, None) == [0, 2, 4, 6, 8]
    assert shares(0, 3, None) == [0, 0, 0, 0]
    assert shares(5, 3, [0, 0, 5, 5]) == [0, 0, 5, 5]
    for rows, n, splits in ((7, 2, None), (4, 0, None), (4, 128, None), (4, 2, [0, 4]), (4, 2, [0, 5, 4]), (4, 2, [1, 2, 4]),
                            (4, 2, [])):
        with pytest.raises(ValueError):
            shares(rows, n, splits)


def test_rows_of_a_tensor(lib):
    rows = layers._load().rows_of
    x = torch.zeros(6, 10)
    assert rows(x) == (6, 10, 10)
    assert rows(x[:, 2:7]) == (6, 5, 10)
    assert rows(x[::2]) == (3, 10, 20)
    assert rows(x.view(2, 3, 10)) == (6, 10, 10)
    assert rows(x.view(2, 3, 10)[:, :, :4]) == (6, 4, 10)
    assert rows(x.view(3, 1, 2, 10)[:, :, :, 1:]) == (6, 9, 10)
    assert rows(x[:1, ::1]) == (1, 10, 10)
    assert rows(torch.zeros(0, 10)) == (0, 10, 10)
    for bad in (x.t(), x[:, ::2], x[0].expand(6, 10), x.view(2, 3, 10)[:, :2], torch.zeros(4, 0), torch.tensor(1.0),
                x.view(2, 3, 10).transpose(0, 1)):
        with pytest.raises(ValueError):
            rows(bad)


def test_binding_refuses_to_run_without_library(lib, tmp_path, monkeypatch):
    monkeypatch.setattr(L, "LIB_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(L, "_lib", None)
    monkeypatch.setattr(layers, "_native", None)
    with pytest.raises(RuntimeError, match="missing"):
        layers.embedding_forward(torch.zeros(2, 2), torch.zeros(1, dtype=torch.int64))


# ---------------------------------------------------------------- GPU parity
def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, mean=0.0, dtype=F32):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def padded(t, extra, offset=0):
    """The same rows in a buffer with longer rows, starting at a column."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[:, offset:offset + t.shape[1]]
    view.copy_(t)
    return view


def token_ids(g, n, vocab, kind, dtype=torch.int64):
    if kind == "same":
        ids = torch.full((n,), vocab - 1, device="cuda")
    elif kind == "zipf":
        ids = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab + 1)).long() - 1
    else:
        ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ids = ids.clamp(0, vocab - 1)
    if kind == "padded":
        far = torch.tensor([-1, vocab, -(1 << 31), (1 << 31) - 1], device="cuda")
        at = torch.rand(n, generator=g, device="cuda") < 0.3
        ids = torch.where(at, far[torch.randint(0, 4, (n,), generator=g, device="cuda")], ids)
        if dtype == torch.int64 and n > 2:
            ids[n // 2] = 1 << 40
    if kind == "dense":  # but for the first 4096, few ids
        ids[4096:] %= 1 + vocab // 1000
    if kind == "none":
        ids = torch.full((n,), -1, device="cuda")
    return ids.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("table_dtype,dtype", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("n,vocab,cols,extra", [(1, 1, 1, 0), (7, 5, 3, 0), (33, 100, 6, 0), (48, 300, 768, 0), (5, 40, 768, 8),
                                                (9, 33, 1000, 1), (3, 20, 4096, 0), (257, 64, 64, 0), (2, 9, 5000, 4),
                                                (2, 9, 9001, 0)])
@pytest.mark.parametrize("ids_dtype", [torch.int32, torch.int64])
def test_embedding_forward(cuda_lib, table_dtype, dtype, n, vocab, cols, extra, ids_dtype):
    g = gen(n * 7 + cols)
    table = padded(normal(g, vocab, cols, dtype=table_dtype), extra)
    ids = token_ids(g, n, vocab, "padded", ids_dtype)
    scale = 3.0
    y = layers.embedding_forward(table, ids, scale=scale, dtype=dtype)
    out = padded(torch.zeros(n, cols, dtype=dtype, device="cuda"), extra)
    layers.embedding_forward(table, ids, scale=scale, dtype=dtype, out=out)
    assert torch.equal(out, y)
    if extra:
        assert out._base.isnan().sum() == n * extra     # what lies between the rows stays
    inside = (ids >= 0) & (ids < vocab)
    ref = torch.where(inside[:, None], table.double()[torch.where(inside, ids, 0).long()] * scale, 0.0)
    # One fp32 product, one rounding to the output's type.
    assert ((y.double() - ref).abs() <= ref.abs() * (U + half(dtype) * (1 + U))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,ld", [(1, 1), (3, 3), (7, 9), (8, 8), (17, 17), (33, 34), (130, 131), (515, 515), (1026, 1026)])
def test_embedding_forward_any_address(cuda_lib, dtype, cols, ld):
    """Tables and outputs at every place within 16 bytes, and rows up to the
    ends of their buffers: what lies around them is left as it was."""
    g = gen(cols)
    vocab, n, per = 23, 41, 16 // dtype.itemsize
    ids = token_ids(g, n, vocab, "padded")
    ids[:4] = torch.tensor([0, vocab - 1, 1, vocab - 2], device="cuda")
    inside = (ids >= 0) & (ids < vocab)
    for a in range(per):
        for b in range(per):
            table = normal(g, a + (vocab - 1) * ld + cols, dtype=dtype)[a:].as_strided((vocab, cols), (ld, 1))
            buf = torch.full((b + n * ld + 16,), 7.0, dtype=dtype, device="cuda")
            out = buf[b:].as_strided((n, cols), (ld, 1))
            want = buf.clone()
            for scale in (1.0, -0.5):
                want[b:].as_strided((n, cols), (ld, 1)).copy_(torch.where(inside[:, None], table[ids.where(inside, 0)] * scale, 0.0))
                layers.embedding_forward(table, ids, scale=scale, out=out)
                assert torch.equal(buf, want), (a, b, scale)


def embedding_reference(ids, dy, vocab, splits, scale):
    """Gradients and the sums of their terms' magnitudes, and counts."""
    out = []
    for a, b in zip(splits, splits[1:]):
        i, d = ids[a:b].long(), dy[a:b].double() * scale
        at = torch.nonzero((i >= 0) & (i < vocab))[:, 0]
        g = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
        mag, cnt = torch.zeros_like(g), torch.zeros(vocab, dtype=torch.float64, device="cuda")
        g.index_put_((i[at],), d[at], accumulate=True)
        mag.index_put_((i[at],), d[at].abs(), accumulate=True)
        cnt.index_put_((i[at],), torch.ones(len(at), dtype=torch.float64, device="cuda"), accumulate=True)
        out.append((g, mag, cnt[:, None]))
    return out


EMBED_BACKWARD = [
    # rows by worker, vocab, columns, ids, extra columns of dy
    ([1], 1, 1, "uniform", 0),
    ([0], 3, 4, "uniform", 0),
    ([5, 0, 3], 7, 3, "uniform", 0),
    ([64, 64], 50, 64, "same", 0),
    ([31, 33, 32], 5, 8, "padded", 0),
    ([100], 1000, 768, "none", 0),
    ([1000, 1, 95], 300, 256, "zipf", 8),
    ([4096], 513, 40, "uniform", 0),
    ([4097, 12289], 60000, 24, "zipf", 0),
    ([20000], 3, 17, "uniform", 1),
    ([40000], 70000, 8, "zipf", 0),             # ten sorted tiles: a merge
    ([270000, 7], 263000, 4, "zipf", 0),        # more than 32: two
    ([130000, 9000], 60000, 4, "dense", 0),     # what a block looks through does not fit shared memory
    ([9000], 1, 300, "same", 0),
    ([700] * 9, 128, 770, "zipf", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dy_dtype,dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("shares,vocab,cols,kind,extra", EMBED_BACKWARD)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward(cuda_lib, dy_dtype, dtype, shares, vocab, cols, kind, extra, accumulate):
    splits = [0]
    for s in shares:
        splits.append(splits[-1] + s)
    n, scale = splits[-1], 1.5
    g = gen(n + vocab + cols)
    dy = padded(normal(g, n, cols, dtype=dy_dtype), extra)
    ids = token_ids(g, n, vocab, kind, torch.int32 if cols % 2 else torch.int64)
    if accumulate:
        old = [normal(g, vocab, cols, dtype=dtype) for _ in shares]
        grads = [o.clone() for o in old]
        got = layers.embedding_backward(ids, dy, vocab, len(shares), splits, scale, dtype, out=grads, accumulate=True)
        assert all(a is b for a, b in zip(got, grads))
    else:
        # A buffer one element past a 16-byte boundary takes the narrow path.
        wide = layers.embedding_backward(ids, dy, vocab, len(shares), splits, scale, dtype)
        off = [torch.full((vocab * cols + 1,), float("nan"), dtype=dtype, device="cuda")[1:].view(vocab, cols) for _ in shares]
        got = layers.embedding_backward(ids, dy, vocab, len(shares), splits, scale, dtype, out=off)
        assert all(torch.equal(a, b) for a, b in zip(got, wide))
    for m, (ref, mag, cnt) in enumerate(embedding_reference(ids, dy, vocab, splits, scale)):
        r = got[m].double()
        if accumulate:
            untouched = (cnt == 0)[:, 0]
            assert torch.equal(got[m][untouched], old[m][untouched])
            ref, mag = ref + old[m].double(), mag + old[m].double().abs()
        # cnt sums, the product with scale (one more for old + it), the output's rounding.
        bound = (cnt + 2) * U * mag + half(dtype) * (ref.abs() + (cnt + 2) * U * mag)
        assert ((r - ref).abs() <= bound).all(), m


@pytest.mark.gpu
def test_embedding_gradient_against_differences(cuda_lib):
    """d/dW of sum(y * c) by central differences of the forward call, in a
    function that is linear in W: exact up to the fp32 roundings of y."""
    g = gen(3)
    table, ids = normal(g, 5, 3), torch.tensor([1, 4, 1, -1, 0, 1], device="cuda")
    c = normal(g, 6, 3)
    grad = layers.embedding_backward(ids, c, 5, scale=2.0)[0].double()
    for v in range(5):
        for j in range(3):
            hi, lo = table.clone(), table.clone()
            hi[v, j] += 0.5
            lo[v, j] -= 0.5
            d = sum(s * (layers.embedding_forward(t, ids, scale=2.0).double() * c.double()).sum() for s, t in ((1, hi), (-1, lo)))
            step = hi[v, j].double() - lo[v, j].double()
            # y differs by at most u |y| on both sides, y up to 2 (|W| + 0.5); the gradient itself by its 3-term sum.
            bound = 4 * U * 2 * (table.abs().max().double() + 0.5) * c.double().abs().sum() + 8 * U * c.double().abs().sum()
            assert abs(d / step - grad[v, j]) <= bound


NORM = [  # rows by worker, columns, extra columns
    ([1], 1, 0), ([2, 0, 5], 2, 0), ([3], 7, 0), ([8, 9], 64, 0), ([64], 768, 0), ([70, 1, 29], 768, 8), ([37], 1000, 0),
    ([16, 16], 999, 0), ([20], 1026, 1), ([9], 2304, 0), ([7, 6], 4096, 0), ([5], 4098, 0), ([3], 8192, 0), ([4, 3], 9001, 0),
    ([3], 16384, 0), ([2, 3], 20000, 0), ([1], 33001, 2), ([0], 64, 0), ([3000, 1000], 48, 0), ([2000] * 5, 96, 0),
]


def norm_inputs(shares, cols, extra, dtype, w_dtype, seed=0):
    n = sum(shares)
    g = gen(seed + n * 3 + cols)
    x = padded(normal(g, n, cols, std=2.0, mean=1.0, dtype=dtype), extra)
    w = normal(g, cols, std=0.2, mean=1.0, dtype=w_dtype)
    b = normal(g, cols, dtype=w_dtype)
    return g, x, w, b, even(n, 1)[:1] + [sum(shares[:i + 1]) for i in range(len(shares))]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,w_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("shares,cols,extra", NORM)
@pytest.mark.parametrize("bias", [False, True])
def test_layer_norm_forward(cuda_lib, dtype, w_dtype, shares, cols, extra, bias):
    g, x, w, b, _ = norm_inputs(shares, cols, extra, dtype, w_dtype)
    eps = 1e-5
    y, mean, rstd = layers.layer_norm_forward(x, w, b if bias else None, eps)
    X = x.double()
    mu = X.mean(1)
    var = (X - mu[:, None]).square().mean(1)
    r = (var + eps).rsqrt()
    # A sum goes through at most 16 elements of a thread (cols / 512 where a
    # row does not fit a block's registers), 5 + 32 joins of lanes and warps.
    depth = 64 + cols / 512
    e_mu = depth * U * X.abs().mean(1) + U * mu.abs()
    # Relative: the squares' sum, the mean's own error against the deviation,
    # and a few ulps of the reciprocal square root (2 of rsqrtf).
    e_r = (depth + 8) * U + 2 * e_mu * r
    assert ((mean.double() - mu).abs() <= e_mu).all()
    assert ((rstd.double() - r).abs() <= e_r * r).all()
    xh = (X - mu[:, None]) * r[:, None]
    B = b.double() if bias else torch.zeros_like(w).double()
    ref = xh * w.double() + B
    e_xh = (e_mu * r)[:, None] + (e_r[:, None] + 3 * U) * xh.abs()
    e = e_xh * w.double().abs() + 2 * U * ((xh * w.double()).abs() + B.abs())
    assert ((y.double() - ref).abs() <= e + half(dtype) * (ref.abs() + e)).all()
    inplace = x.clone()
    layers.layer_norm_forward(inplace, w, b if bias else None, eps, out=inplace)
    # The clone has no gaps between its rows, so another width of loads may
    # have been taken, and with it another order of the sums.
    assert ((inplace.double() - ref).abs() <= e + half(dtype) * (ref.abs() + e)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,w_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("shares,cols,extra", NORM)
@pytest.mark.parametrize("bias", [False, True])
def test_layer_norm_backward(cuda_lib, dtype, w_dtype, shares, cols, extra, bias):
    g, x, w, _, splits = norm_inputs(shares, cols, extra, dtype, w_dtype, seed=5)
    n = splits[-1]
    dy = padded(normal(g, n, cols, dtype=dtype), extra)
    _, mean, rstd = layers.layer_norm_forward(x, w)
    dx, dw, db = layers.layer_norm_backward(dy, x, w, mean, rstd, len(shares), splits, bias=bias)
    assert (db is not None) == bias and len(dw) == len(shares)
    # The formula at the given mean and rstd, which are inputs here.
    r, D = rstd.double()[:, None], dy.double()
    xh = (x.double() - mean.double()[:, None]) * r
    e_xh = 2 * U * (xh.abs() + 0)                # a difference and a product
    gy = D * w.double()
    s1, s2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    ref = r * (gy - s1 - xh * s2)
    depth = 64 + cols / 512
    e1 = (depth + 2) * U * gy.abs().mean(1, keepdim=True)
    e2 = (depth + 6) * U * (gy * xh).abs().mean(1, keepdim=True)
    e = r * (U * gy.abs() + e1 + xh.abs() * e2 + 4 * U * (gy.abs() + s1.abs() + (xh * s2).abs()) + e_xh * s2.abs())
    assert ((dx.double() - ref).abs() <= e + half(dtype) * (ref.abs() + e)).all()
    for m, (a, b) in enumerate(zip(splits, splits[1:])):
        t = D[a:b] * xh[a:b]
        # Rows are added one after another within a group of threads, groups
        # and blocks (each at most the number of rows) after them.
        k = (b - a) + 8
        for got, ref, mag in ((dw[m], t.sum(0), t.abs().sum(0)), (db[m], D[a:b].sum(0), D[a:b].abs().sum(0))) if bias else \
                ((dw[m], t.sum(0), t.abs().sum(0)),):
            e = (k + 4) * U * mag
            assert got.dtype == w_dtype and got.shape == w.shape
            assert ((got.double() - ref).abs() <= e + half(w_dtype) * (ref.abs() + e)).all(), m
    again = layers.layer_norm_backward(dy, x, w, mean, rstd, len(shares), splits, bias=bias)
    assert torch.equal(again[0], dx) and all(torch.equal(p, q) for p, q in zip(again[1], dw))
    inplace = dy.clone()
    _, dw2, db2 = layers.layer_norm_backward(inplace, x, w, mean, rstd, len(shares), splits, bias=bias, out=inplace)
    for m, (a, b) in enumerate(zip(splits, splits[1:])):
        t = D[a:b] * xh[a:b]
        for got, want, mag in ((dw2[m], t.sum(0), t.abs().sum(0)), (db2[m], D[a:b].sum(0), D[a:b].abs().sum(0))) if bias else \
                ((dw2[m], t.sum(0), t.abs().sum(0)),):
            e = (b - a + 12) * U * mag
            assert ((got.double() - want).abs() <= e + half(w_dtype) * (want.abs() + e)).all(), m
    e = r * (U * gy.abs() + e1 + xh.abs() * e2 + 4 * U * (gy.abs() + s1.abs() + (xh * s2).abs()) + e_xh * s2.abs())
    ref = r * (gy - s1 - xh * s2)
    assert ((inplace.double() - ref).abs() <= e + half(dtype) * (ref.abs() + e)).all()


@pytest.mark.gpu
def test_layer_norm_gradient_against_differences(cuda_lib):
    """sum(y c) over x by central differences of the forward call."""
    g = gen(11)
    x, w, b, c = normal(g, 2, 6, std=2.0), normal(g, 6, mean=1.0), normal(g, 6), normal(g, 2, 6)
    _, mean, rstd = layers.layer_norm_forward(x, w, b)
    dx, dw, db = layers.layer_norm_backward(c, x, w, mean, rstd)
    f = lambda x_, w_, b_: float((layers.layer_norm_forward(x_, w_, b_)[0].double() * c.double()).sum())  # noqa: E731
    h = 2.0 ** -6
    # Truncation: h^2 / 6 times the third derivative, of the order of
    # sum |c w| 15 r^3 for a normalised row; rounding: 64 u sum |c y| / h.
    y = layers.layer_norm_forward(x, w, b)[0].double()
    scale = float((c.double() * w.double()).abs().sum())
    bound = h * h / 6 * 15 * scale * float(rstd.max()) ** 3 + 64 * U * float((c.double() * y).abs().sum() + scale) / h
    for arg, grad in ((x, dx), (w, dw[0]), (b, db[0])):
        flat, gflat = arg.view(-1), grad.view(-1)
        for i in range(flat.numel()):
            old = flat[i].item()
            flat[i] = old + h
            hi = f(x, w, b)
            flat[i] = old - h
            lo = f(x, w, b)
            flat[i] = old
            assert abs((hi - lo) / (2 * h) - float(gflat[i])) <= bound


@pytest.mark.gpu
def test_layer_norm_nan_row_stays_in_its_row(cuda_lib):
    g, x, w, b, _ = norm_inputs([40], 768, 0, BF16, BF16)
    clean = layers.layer_norm_forward(x, w, b)
    x[3, 5], x[7, 0], x[9, 700] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = layers.layer_norm_forward(x, w, b)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 7, 9]] = True
    assert y[bad].isnan().all() and rstd[bad].isnan().all()
    for a, c in zip((y, mean, rstd), clean):
        assert torch.equal(a[~bad], c[~bad])


# ------------------------------------------------------------- distillation
def distill_inputs(shares, vocab, top, dtype, kind, seed=0, extra=0, top_dtype=F32, ids_dtype=torch.int64):
    n = sum(shares)
    g = gen(seed + n * 5 + vocab + top)
    z = normal(g, n, vocab, std=2.0, dtype=dtype)
    u = normal(g, n, top, std=1.5, dtype=top_dtype)
    ids = torch.rand(n, vocab, generator=g, device="cuda").topk(min(top, vocab), dim=1).indices if vocab <= 20000 else \
        torch.randint(0, vocab, (n, top), generator=g, device="cuda")
    if ids.shape[1] < top or kind == "twice":
        ids = torch.randint(0, max(1, min(vocab, top // 2)), (n, top), generator=g, device="cuda")
    if kind == "holes":
        z[:, vocab - vocab // 8:] = -math.inf                  # a padded vocabulary
        if vocab > 8:
            ids[ids >= vocab - vocab // 8] = -1
        ids[torch.rand(n, top, generator=g, device="cuda") < 0.2] = vocab
        u[torch.rand(n, top, generator=g, device="cuda") < 0.2] = -math.inf
        dead = torch.rand(n, generator=g, device="cuda") < 0.3
        ids[dead] = -1
        z[dead] = float("nan")                                 # ignored rows are not looked at
        u[dead] = float("nan")
    return padded(z, extra), ids.to(ids_dtype), u, [sum(shares[:i]) for i in range(len(shares) + 1)]


def distill_reference(z, ids, u, splits, t):
    ids, vocab = ids.long(), z.shape[1]
    here = (ids >= 0) & (ids < vocab) & (u != -math.inf)
    on = here.any(1)
    Z = torch.where(on[:, None], z.double(), 0.0)
    logp = torch.log_softmax(torch.where(here, u.double() / t, -math.inf).masked_fill(~on[:, None], 0.0), 1)
    logq = torch.log_softmax(Z / t, 1)
    safe = torch.where(here, ids, 0)
    terms = torch.where(here, logp.exp() * (logp - logq.gather(1, safe)), 0.0)
    row = terms.sum(1) * t * t
    p = torch.zeros_like(logq).scatter_add_(1, safe, torch.where(here, logp.exp(), 0.0))
    loss, dz = [], torch.zeros_like(logq)
    for a, b in zip(splits, splits[1:]):
        k = int(on[a:b].sum())
        loss.append(row[a:b].sum() / max(k, 1))
        if k:
            dz[a:b] = torch.where(on[a:b, None], (logq[a:b].exp() - p[a:b]) * t / k, 0.0)
    return torch.stack(loss), row, dz, logq, p, on


def check_distill(z, ids, u, splits, t, top):
    n_workers = len(splits) - 1
    loss, row, dz = layers.distill_loss_and_grad(z, ids, u, n_workers, splits, temperature=t)
    loss2, row2 = layers.distill_loss(z, ids, u, n_workers, splits, temperature=t)
    L_, R, D, logq, p, on = distill_reference(z, ids, u, splits, t)
    spread = torch.where(on, (torch.where(on[:, None], z.double(), 0.0).amax(1) - torch.where(
        on[:, None] & z.isfinite(), z.double(), math.inf).amin(1)).clamp(min=0) / t, 0.0)
    uu = u.double() / t
    uspread = torch.where(on, torch.where(u.isfinite(), uu, -math.inf).amax(1) - torch.where(u.isfinite(), uu, math.inf).amin(1), 0.0)
    # Exponentials: 2^-22 of ex2 (2 ulps of expf), the argument's roundings
    # (difference, product; 1 / T) times its size, and the sum: at most
    # vocab / 256 + 64 terms one after another, all positive.
    depth = z.shape[1] / 256 + 64
    e_q = (4 * spread + 8 + depth) * U
    e_p = (4 * uspread + 8 + top) * U
    size = (p * logq.clamp(min=-1e30).abs()).sum(1) + torch.special.entr(p).sum(1).abs()
    e_row = t * t * (e_q + e_p + (e_p + 8 * U) * size + top * U * (size + spread) + 8 * U * (spread + 1))
    for r in (row, row2):
        assert ((r.double() - R).abs() <= e_row + U * R.abs()).all()
    assert not (row[~on] != 0).any() and not (dz[~on] != 0).any()
    for m, (a, b) in enumerate(zip(splits, splits[1:])):
        k = max(int(on[a:b].sum()), 1)
        bound = e_row[a:b].sum() / k + 2 * U * R[a:b].abs().sum() / k
        assert abs(loss[m].double() - L_[m]) <= bound and abs(loss2[m].double() - L_[m]) <= bound
        c = t / k
        e = c * ((e_q[a:b, None] + 4 * U) * logq[a:b].exp() + (e_p[a:b, None] + 4 * U) * p[a:b])
        assert ((dz[a:b].double() - D[a:b]).abs() <= e + half(z.dtype) * (D[a:b].abs() + e) + 2.0 ** -126).all(), m
    return loss, row, dz


DISTILL = [  # rows by worker, vocab, top, kind, extra columns
    ([1], 1, 1, "plain", 0), ([2], 2, 3, "twice", 0), ([3, 0, 4], 33, 5, "holes", 0), ([5], 1000, 64, "plain", 0),
    ([4, 4], 1001, 20, "holes", 0), ([6], 4096, 33, "holes", 8), ([3], 32001, 8, "plain", 0), ([2, 3], 50000, 64, "holes", 0),
    ([3], 50001, 128, "holes", 3), ([2], 131101, 20, "plain", 0), ([2], 300, 1024, "twice", 0), ([2, 2], 60000, 1000, "plain", 0),
    ([300, 100], 200, 16, "holes", 0), ([0], 50, 4, "plain", 0), ([2], 200000, 7, "holes", 1), ([400], 3001, 40, "plain", 0),
    # A warp a row, several rows a warp, workers that begin within a block; and
    # the shortest rows that blocks take.
    ([20000, 0, 37, 5], 33, 3, "holes", 0), ([9], 129, 40, "twice", 1), ([40, 3], 1024, 70, "holes", 0),
    ([30, 2], 1025, 300, "holes", 0), ([17, 31, 250], 1500, 5, "holes", 0), ([1500], 5000, 6, "holes", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,top_dtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("shares,vocab,top,kind,extra", DISTILL)
@pytest.mark.parametrize("temperature", [1.0, 0.5, 4.0])
def test_distill(cuda_lib, dtype, top_dtype, shares, vocab, top, kind, extra, temperature):
    z, ids, u, splits = distill_inputs(shares, vocab, top, dtype, kind, extra=extra, top_dtype=top_dtype,
                                       ids_dtype=torch.int32 if top % 2 else torch.int64)
    loss, row, dz = check_distill(z, ids, u, splits, temperature, top)
    n = len(shares)
    again = layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=temperature)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, row, dz)))
    # Over the logits, and into rows of another alignment.
    over = z.clone() if not extra else padded(z, extra)
    got = layers.distill_loss_and_grad(over, ids, u, n, splits, temperature=temperature, out=over)
    other = padded(torch.zeros(z.shape, dtype=dtype, device="cuda"), 3, offset=1)
    layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=temperature, out=other)
    tol = half(dtype) * 2 + 2.0 ** -18
    for t in (got[2], other):
        d = (t.double() - dz.double()).abs()
        assert (d <= tol * dz.double().abs() + 2.0 ** -18 * temperature).all()
    if other.numel():
        assert other._base[:, 0].isnan().all() and other._base[:, -2:].isnan().all()
    double = layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=temperature, grad_scale=2.0)[2]
    assert torch.equal(double, dz * 2)           # powers of two change no rounding


@pytest.mark.gpu
def test_distill_extreme_logits(cuda_lib):
    """Finite masks of the type's lowest value, large logits, and what is not finite."""
    for dtype, vocab in itertools.product((F32, BF16), (300, 3000)):
        z, ids, u, splits = distill_inputs([6], vocab, 8, dtype, "plain")
        lowest = torch.finfo(dtype).min
        z[0, 100:] = lowest
        ids[0] = torch.arange(8, device="cuda")
        z[1] = 1e4
        z[2, 7] = 3e4
        u[3] = lowest if dtype == F32 else -1e30     # equal lowest entries share the mass
        u[4, 1:] = -1e30
        check_distill(z, ids, u, splits, 1.0, 8)
        check_distill(z, ids, u, splits, 0.5, 8)
        z[1, 5], z[2, 5], u[3, 2] = float("nan"), float("inf"), float("nan")
        z[4] = float("-inf")
        clean = [0, 5]
        ref = layers.distill_loss_and_grad(z[clean].contiguous(), ids[clean].contiguous(), u[clean].contiguous())
        _, row, dz = layers.distill_loss_and_grad(z, ids, u)
        assert row[1:5].isnan().all() and dz[1:5].isnan().any(1).all()
        assert torch.equal(row[clean], ref[1])
        # A present entry whose student logit is -inf: the loss is inf, the gradient finite.
        z, ids, u, _ = distill_inputs([1], vocab, 8, F32, "plain")
        z[0, ids[0, 2]] = float("-inf")
        loss, row, dz = layers.distill_loss_and_grad(z, ids, u)
        assert row[0] == math.inf and loss[0] == math.inf and dz.isfinite().all()


@pytest.mark.gpu
def test_distill_gradient_against_differences(cuda_lib):
    g = gen(21)
    z, u = normal(g, 3, 10), normal(g, 3, 4)
    ids = torch.tensor([[0, 3, 3, 9], [-1, 2, 5, 6], [-1, -1, -1, -1]], device="cuda")
    t, h = 2.0, 2.0 ** -5
    dz = layers.distill_loss_and_grad(z, ids, u, temperature=t)[2]
    f = lambda: float(layers.distill_loss(z, ids, u, temperature=t)[0][0])  # noqa: E731
    # Third derivative of log sum exp(z / T) by one logit: at most 1 / T^3 (times T^2);
    # a loss of at most 10 is off by at most 2^7 u.
    bound = h * h / 6 / t + 10 * 2.0 ** 7 * U / h
    for n in range(3):
        for v in range(10):
            old = z[n, v].item()
            z[n, v] = old + h
            hi = f()
            z[n, v] = old - h
            lo = f()
            z[n, v] = old
            assert abs((hi - lo) / (2 * h) - float(dz[n, v])) <= bound


# ------------------------------------------------------------- as they are used
@pytest.mark.gpu
def test_other_streams_and_graphs(cuda_lib):
    """Two captured graphs and eager calls, interleaved on several streams,
    give what each gives alone."""
    def inputs(seed):
        g = gen(seed)
        ids = token_ids(g, 600, 97, "zipf")
        x = normal(g, 600, 97, std=2.0)
        return ids, x, normal(g, 97, mean=1.0), normal(g, 600, 5), torch.randint(0, 97, (600, 5), generator=g, device="cuda")

    def calls(ids, x, w, u, top):
        y, mean, rstd = layers.layer_norm_forward(x, w)
        loss, row, dz = layers.distill_loss_and_grad(y, top, u, 3)
        dx, dw, db = layers.layer_norm_backward(dz, x, w, mean, rstd, 3)
        return [layers.embedding_forward(x[:97], ids), y, loss, row, dz, dx, *dw, *db,
                *layers.embedding_backward(ids, dx, 97, 3)]
    sets = [inputs(s) for s in range(3)]
    alone = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets[:2]:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(calls(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = calls(*sets[2])
    torch.cuda.synchronize()
    for got, want in zip((*outs, eager), alone):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_refused_tensors(cuda_lib):
    x = torch.zeros(4, 8, device="cuda")
    w, ids = x[0].clone(), torch.zeros(4, dtype=torch.int64, device="cuda")
    top, u = ids.view(4, 1), x[:, :1].contiguous()
    bad = [
        (ValueError, lambda: layers.embedding_forward(x[0], ids)),
        (TypeError, lambda: layers.embedding_forward(x.half(), ids)),
        (TypeError, lambda: layers.embedding_forward(x, ids.short())),
        (ValueError, lambda: layers.embedding_forward(x, ids[::2])),
        (ValueError, lambda: layers.embedding_forward(x.t(), ids)),
        (ValueError, lambda: layers.embedding_forward(x, ids, out=x[:, :4])),
        (TypeError, lambda: layers.embedding_forward(x, ids, out=x.bfloat16())),
        (ValueError, lambda: layers.embedding_backward(ids[:3], x, 8)),
        (ValueError, lambda: layers.embedding_backward(ids, w.expand(4, 8), 8)),
        (ValueError, lambda: layers.embedding_backward(ids, x, 8, n_workers=3)),
        (ValueError, lambda: layers.embedding_backward(ids, x, 8, accumulate=True)),
        (ValueError, lambda: layers.embedding_backward(ids, x, 4, n_workers=2, out=[x])),
        (ValueError, lambda: layers.embedding_backward(ids, x, 4, out=[torch.zeros(8, 4, device="cuda").t()])),
        (ValueError, lambda: layers.embedding_backward(ids, x, 0)),
        (ValueError, lambda: layers.embedding_backward(ids, x, 2, n_workers=2, out=[x[:2], x[1:3]])),
        (ValueError, lambda: layers.embedding_backward(ids, x, 2, n_workers=2, out=[x[:2], x[:2]])),
        (ValueError, lambda: layers.embedding_forward(x, ids, out=x)),
        (ValueError, lambda: layers.embedding_backward(ids, x, 4, out=[x])),
        (ValueError, lambda: layers.layer_norm_forward(x[:3], w, out=x[1:])),
        (ValueError, lambda: layers.layer_norm_backward(x[:3], x[:3].clone(), w, w[:3], w[:3], out=x[1:])),
        (ValueError, lambda: layers.layer_norm_backward(x.clone(), x, w, w[:4], w[:4], out=x)),
        (ValueError, lambda: layers.distill_loss_and_grad(x[:3], top[:3], u[:3], out=x[1:])),
        (ValueError, lambda: layers.layer_norm_forward(x, w[:7])),
        (TypeError, lambda: layers.layer_norm_forward(x, w, w.bfloat16())),
        (ValueError, lambda: layers.layer_norm_forward(x, w, eps=-1.0)),
        (ValueError, lambda: layers.layer_norm_forward(x, w.cpu())),
        (TypeError, lambda: layers.layer_norm_backward(x.bfloat16(), x, w, w[:4], w[:4])),
        (ValueError, lambda: layers.layer_norm_backward(x, x, w, w[:3], w[:4])),
        (TypeError, lambda: layers.layer_norm_backward(x, x, w, w[:4].double(), w[:4])),
        (ValueError, lambda: layers.distill_loss(x, top[:3], u)),
        (ValueError, lambda: layers.distill_loss(x, top, torch.zeros(4, 2, device="cuda"))),
        (ValueError, lambda: layers.distill_loss(x, top, u, temperature=0.0)),
        (ValueError, lambda: layers.distill_loss(x, top.expand(4, 2), u.expand(4, 2))),
        (ValueError, lambda: layers.distill_loss(x, top.repeat(1, 1025), u.repeat(1, 1025))),
        (ValueError, lambda: layers.distill_loss_and_grad(x, top, u, out=x[:, :4])),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_training_step_with_the_optimizer(cuda_lib, dtype):
    """tokens -> embedding -> norm -> tied output layer -> distillation and
    back, with one gradient per worker for every weight, into the Signum step;
    each worker's gradients against autograd's on that worker's rows alone."""
    workers, rows, vocab, d, top = 3, 96, 160, 64, 6
    g = gen(31)
    table = normal(g, vocab, d, std=0.5, dtype=dtype)
    w, b = normal(g, 1, d, std=0.1, mean=1.0, dtype=dtype), normal(g, 1, d, std=0.1, dtype=dtype)
    ids = token_ids(g, rows, vocab, "zipf")
    top_ids = torch.rand(rows, vocab, generator=g, device="cuda").topk(top, dim=1).indices
    top_ids[::7] = -1
    u = normal(g, rows, top)
    splits, scale, t = [0, 30, 61, rows], 2.0, 2.0

    x = layers.embedding_forward(table, ids, scale)
    y, mean, rstd = layers.layer_norm_forward(x, w, b)
    loss, _, dz = layers.distill_loss_and_grad(y @ table.t(), top_ids, u, workers, splits, temperature=t)
    dy = dz @ table
    dx, dw, db = layers.layer_norm_backward(dy, x, w, mean, rstd, workers, splits)
    tied = [dz[a:c].t() @ y[a:c] for a, c in zip(splits, splits[1:])]
    grads = layers.embedding_backward(ids, dx, vocab, workers, splits, scale, out=tied, accumulate=True)

    u_out = half(dtype)
    for m, (a, c) in enumerate(zip(splits, splits[1:])):
        T, W, B = (q.double().requires_grad_() for q in (table, w, b))
        X = T[ids[a:c]] * scale
        Y = torch.nn.functional.layer_norm(X, (d,), W[0], B[0], 1e-5)
        here = top_ids[a:c] >= 0
        logp = torch.log_softmax(u[a:c].double() / t, 1)
        logq = torch.log_softmax(Y @ T.t() / t, 1).gather(1, top_ids[a:c].clamp(min=0))
        ref = (torch.where(here, logp.exp() * (logp - logq), 0.0).sum() * t * t) / here.any(1).sum()
        ref.backward()
        # Six roundings to the type on the way (x, y, logits, dz, dy, dx), in
        # norm, each at most u_out of what it rounds, amplified by sums of the
        # layers in between by at most sqrt(d): 6 sqrt(64) half steps.
        tol = 6 * math.sqrt(d) * u_out + 1e-5
        assert abs(loss[m].item() - ref.item()) <= tol * abs(ref.item())
        for got, want in ((grads[m], T.grad), (dw[m], W.grad), (db[m], B.grad)):
            assert got.shape == want.shape
            assert (got.double() - want).norm() <= tol * want.norm()

    shapes = [(vocab, d), (1, d), (1, d)]
    opt = SignMuonStep(shapes, workers, 0, "pack1", 0.9, 0.01, dtype)
    weights = [q.clone() for q in (table, w, b)]
    opt.step(weights, [*grads, *dw, *db])
    for i, per_worker in enumerate((grads, dw, db)):
        votes = sum(torch.where(q < 0, -1, 1) for q in per_worker).sign()
        before = (table, w, b)[i].double()
        # One rounding of W - eta vote to the type (eta is an fp32 number).
        eta = float(torch.tensor(0.01))
        expect = before - eta * votes
        assert ((weights[i].double() - expect).abs() <= u_out * expect.abs()).all()
