"""The token operators at the edges of what they accept: extreme logits and
temperatures, buffers that a caller owns, sizes where a cost could run away.

Bounds as in test_layers: U = 2^-24 is the most an fp32 rounding is off,
`half` the same for an output's type."""
import os
import re

import pytest
import torch

from sign_muon_optimizer_momentum_b200 import _lib as L
from sign_muon_optimizer_momentum_b200 import layers
from test_layers import BF16, DISTILL, F32, U, distill_inputs, distill_reference, half, lib, padded  # noqa: F401


def device_ms(f, reps=5):
    """The least time of a call on the device."""
    f()
    best = float("inf")
    for _ in range(reps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        begin.record()
        f()
        end.record()
        end.synchronize()
        best = min(best, begin.elapsed_time(end))
    return best


def distill_bounds(z, u, splits, t, top, ref):
    """What the losses by row and worker and the gradient may be off, from
    check_distill of test_layers.  (A spread counts to 200: what lies further
    below the largest is e^-200 and less, nothing beside it.)"""
    _, R, D, logq, p, on = ref
    inf = float("inf")

    def spread_of(x):
        x = x.double() / t
        d = torch.where(x.isfinite(), x, -inf).amax(1) - torch.where(x.isfinite(), x, inf).amin(1)
        return torch.where(on, d, 0.0).clamp(0.0, 200.0)
    spread, uspread = spread_of(z), spread_of(u)
    e_q = (4 * spread + 8 + z.shape[1] / 256 + 64) * U
    e_p = (4 * uspread + 8 + top) * U
    size = (p * logq.clamp(min=-1e38)).abs().sum(1) + torch.special.entr(p).sum(1).abs()
    e_row = t * t * (e_q + e_p + (e_p + 8 * U) * size + top * U * (size + spread) + 8 * U * (spread + 1)) + U * R.abs()
    e_loss, e_dz = [], torch.zeros_like(D)
    for a, b in zip(splits, splits[1:]):
        k = max(int(on[a:b].sum()), 1)
        e_loss.append((e_row[a:b].sum() + U * R[a:b].abs().sum()) / k)
        e = t / k * ((e_q[a:b, None] + 4 * U) * logq[a:b].exp() + (e_p[a:b, None] + 4 * U) * p[a:b])
        e_dz[a:b] = e + half(z.dtype) * (D[a:b].abs() + e) + 2.0 ** -126
    return torch.stack(e_loss), e_row, e_dz


def check_result(got, ref, bounds):
    """Losses by worker, by row, and the gradient, each within its bound."""
    for what, g, r, e in zip(("loss", "row_loss", "gradient"), got, ref, bounds):
        assert ((g.double() - r).abs() <= e).all(), what


MISALIGNED = [([700, 0, 1, 900, 300], 1100, 5, "holes"), ([1300, 40], 1030, 70, "plain"), ([3], 70001, 9, "twice")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shares,vocab,top,kind", MISALIGNED)
def test_distill_rows_at_any_address(cuda_lib, dtype, shares, vocab, top, kind):
    """Logits off 16 bytes, whose rows a block takes from several workers."""
    z, ids, u, splits = distill_inputs(shares, vocab, top, dtype, kind)
    z = padded(z, 3, offset=1)
    ref = distill_reference(z, ids, u, splits, 2.0)
    bounds = distill_bounds(z, u, splits, 2.0, top, ref)
    check_result(layers.distill_loss_and_grad(z, ids, u, len(shares), splits, temperature=2.0), ref, bounds)
    over = layers.distill_loss_and_grad(z, ids, u, len(shares), splits, temperature=2.0, out=z)
    assert over[2] is z
    check_result(over, ref, bounds)


@pytest.mark.gpu
def test_distill_misaligned_gradient_grows_with_its_rows(cuda_lib):
    """Ten times the rows of one worker take about ten times as long: what a
    row costs does not depend on how many rows its worker has."""
    def ms(n):
        z = padded(torch.zeros(n, 1100, dtype=BF16, device="cuda"), 1, offset=1)
        ids, u = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
        out = torch.empty(n, 1101, dtype=BF16, device="cuda")[:, 1:]
        return device_ms(lambda: layers.distill_loss_and_grad(z, ids, u, out=out))
    assert ms(200000) <= 14 * ms(20000)


def check_distill_calls(z, ids, u, splits, t, top):
    """Losses alone, with the gradient, and with it in the logits' place."""
    n = len(splits) - 1
    t32 = torch.tensor(t).item()                 # the temperature as fp32 has it
    ref = distill_reference(z, ids, u, splits, t32)
    bounds = distill_bounds(z, u, splits, t32, top, ref)
    check_result(layers.distill_loss(z, ids, u, n, splits, temperature=t), ref, bounds)
    got = layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=t)
    check_result(got, ref, bounds)
    again = layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=t)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    check_result(layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=t, out=z), ref, bounds)


LARGE = [  # vocab, rows of one kind, columns before the logits in their buffer (off 16 bytes: another kernel)
    (40, 3, 0), (300, 3, 0), (900, 40, 0), (3000, 2, 0), (3000, 60, 0), (20001, 2, 0), (131101, 1, 0), (1100, 2, 1), (70001, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab,each,offset", LARGE)
@pytest.mark.parametrize("kind", ["plain", "twice"])
def test_distill_rows_of_large_logits(cuda_lib, dtype, vocab, each, offset, kind):
    """Rows at a mask's value from end to end, from the middle on, and with one
    logit far above the others, among ordinary rows."""
    lowest = torch.finfo(dtype).min
    whole = [1e10, -1e10, -1e30, lowest, 3e9, 5e6, 2.5e6, -5e6, -2.5e6]
    part = [-1e9, -1e10, -1e30, lowest, -5e6]
    kinds = len(whole) + len(part) + 4
    z, ids, u, splits = distill_inputs([each * kinds // 2, each * kinds - each * kinds // 2], vocab, 8, dtype, kind)
    for i in range(each):
        rows = z[i * kinds:(i + 1) * kinds]
        for j, v in enumerate(whole):
            rows[j] = v
        for j, v in enumerate(part):
            rows[len(whole) + j, vocab // 2:] = v
        rows[-1, vocab // 3] = 1e10
        rows[-2, vocab // 3] = 5e6
        rows[-3] += 3e6             # spread by the type's steps
        ids[i * kinds + 2 * i % kinds] = -1
    check_distill_calls(padded(z, 3, offset=1) if offset else z, ids, u, splits, 1.0, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [200, 5000])
@pytest.mark.parametrize("temperature,std", [(1e-6, 2.0), (1e-6, 1e-7), (1e-3, 3000.0), (1e6, 1e7)])
def test_distill_temperatures_at_the_ends(cuda_lib, dtype, vocab, temperature, std):
    z, ids, u, splits = distill_inputs([30, 7], vocab, 9, dtype, "plain")
    check_distill_calls((z.float() * (std / 2)).to(dtype), ids, u * std, splits, temperature, 9)


FINE = [  # rows by worker, vocab, columns that are not -inf, entries, columns before the logits in their buffer
    ([5, 6], 64, 64, 64, 0), ([40, 3], 512, 512, 512, 0), ([9], 1024, 1024, 1024, 0), ([7], 300, 300, 20, 0),
    ([6, 5], 1500, 600, 600, 0), ([300], 1100, 1000, 1000, 0), ([7], 5000, 700, 700, 0), ([2], 131101, 900, 900, 0),
    ([5, 4], 1500, 600, 600, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shares,vocab,finite,top,offset", FINE)
@pytest.mark.parametrize("temperature", [9.0, 30.0, 100.0, 1000.0, 1e5])
def test_distill_high_temperatures(cuda_lib, dtype, shares, vocab, finite, top, offset, temperature):
    """Teachers that cover all of the vocabulary that there is, whose divergence
    falls as 1 / T^2, and one that does not.

    In units of T^2: sums of at most 64 terms one after another of exponentials
    off by 4 U, twice, and the teacher's entropy (at most log 1024 < 7 times
    what its p are off), 128 + 7 * 80 < 700 U < 2^-14 in all, of at least 1/16
    where fp32 is used: 2^-10 of it.  Else fp64: values of at most 16 after a
    few hundred roundings of 2^-53, at most 2^-40 for kernel and reference, and a
    rounding to fp32."""
    n, t = sum(shares), temperature
    g = torch.Generator(device="cuda")
    g.manual_seed(n * vocab + top)
    z = torch.randn(n, vocab, generator=g, device="cuda") * 2
    z[:, finite:] = -float("inf")
    z = z.to(dtype)
    ids = torch.rand(n, finite, generator=g, device="cuda").topk(top, dim=1).indices
    u = torch.randn(n, top, generator=g, device="cuda") * 1.5
    if top > 64:
        # One id twice in some rows, an entry short in others.
        ids[::3, 5] = ids[::3, 60]
        ids[1::3, 7] = -1
    ids[n // 2] = -1
    splits = [sum(shares[:i]) for i in range(len(shares) + 1)]
    ref = distill_reference(z, ids, u, splits, t)
    _, R, D, logq, p, on = ref
    e_row = R.abs() * 2.0 ** -10 + t * t * 2.0 ** -40
    low = R / (t * t) < 2.0 ** -4 * (1 - 2.0 ** -9)          # those that fp64 has
    tight = R.abs() * 2 * U + t * t * 2.0 ** -40
    e_row = torch.where(low, tight, e_row)
    _, _, e_dz = distill_bounds(z, u, splits, t, top, ref)
    e_loss = []
    for a, b in zip(splits, splits[1:]):
        k = max(int(on[a:b].sum()), 1)
        e_loss.append((e_row[a:b] + U * R[a:b].abs()).sum() / k)
        exact = (half(dtype) + 2 * U) * D[a:b].abs() + t / k * 2.0 ** -40 * (logq[a:b].exp() + p[a:b]) + 2.0 ** -126
        e_dz[a:b] = torch.where(low[a:b, None], exact, e_dz[a:b])
    bounds = torch.stack(e_loss), e_row, e_dz
    if offset:
        z = padded(z, 3, offset=offset)
    m = len(shares)
    check_result(layers.distill_loss(z, ids, u, m, splits, temperature=t), ref, bounds)
    got = layers.distill_loss_and_grad(z, ids, u, m, splits, temperature=t)
    check_result(got, ref, bounds)
    check_result(layers.distill_loss_and_grad(z, ids, u, m, splits, temperature=t, out=z), ref, bounds)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_against_next_tokens_is_cross_entropy(cuda_lib, dtype):
    """One entry a row at temperature 1; negative targets are ignored."""
    n, vocab = 37, 2001
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    z = (torch.randn(n, vocab, generator=g, device="cuda") * 2).to(dtype)
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    target[::5] = -100
    Z = z.double().requires_grad_()
    ref = torch.nn.functional.cross_entropy(Z, target, ignore_index=-100)
    ref.backward()
    loss, row, dz = layers.distill_loss_and_grad(z, target[:, None].contiguous(), torch.zeros(n, 1, device="cuda"))
    # Sums of at most 64 terms of exponentials off by 4 U and arguments of at most 20 (8 U each).
    bound = (64 + 4 + 8 * 20) * U
    assert abs(loss[0].double() - ref.detach()) <= bound
    q = torch.softmax(Z.detach(), 1) / int((target >= 0).sum())
    assert ((dz.double() - Z.grad).abs() <= bound * q + (half(dtype) + 4 * U) * Z.grad.abs() * (1 + bound)).all()
    assert not dz[::5].any() and not row[::5].any()


def test_layer_norm_workspace_is_of_the_size_of_the_call(lib):
    """No more partial rows than the call has rows for, or one for each SM and
    worker where a row is wider than registers hold (148 SMs without a GPU)."""
    size = L.signmuon_layer_norm_backward_workspace_bytes
    for cols in (1, 768, 8192, 16384, 1 << 20):
        row = 2 * 4 * cols
        assert size(cols, [0, 1]) <= 8 * row + 512 + 256
        assert size(cols, [0, 3, 3, 5]) <= (5 + 2 * 7) * row + 512
        assert size(cols, [0, 0]) <= 512
        rows = [0, 1 << 20, 1 << 21]
        assert size(cols, rows) <= (148 * (8 if cols <= 8192 else 1) + 16) * row + 512
    assert size(1 << 20, [0, 1]) <= (8 << 20) + 512


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 7, 64, 999, 2304, 8192, 8193, 20000])
@pytest.mark.parametrize("shares", [[1], [2, 0, 1], [9, 30], [700] * 9, [60000 // 7] * 7])
def test_workspaces_end_where_they_are_said_to(cuda_lib, dtype, cols, shares):
    """Through the C ABI, with workspaces of exactly the size asked for: what
    lies behind them stays."""
    if sum(shares) * cols > 1 << 26:
        shares = shares[:2]
    rows = [sum(shares[:i]) for i in range(len(shares) + 1)]
    n, m, code = rows[-1], len(shares), 0 if dtype == F32 else 1
    g = torch.Generator(device="cuda")
    g.manual_seed(cols + n)
    x, dy = (torch.randn(n, cols, generator=g, device="cuda").to(dtype) for _ in range(2))
    w, stat = torch.ones(cols, dtype=dtype, device="cuda"), torch.ones(n, device="cuda")

    def workspace(size):
        buf = torch.full(((size + 3) // 4 * 4 + 8192,), 77, dtype=torch.uint8, device="cuda")
        return buf, lambda: bool((buf[size:] == 77).all())
    stream = torch.cuda.current_stream().cuda_stream
    for ld in (cols, cols + 1):
        def rows_of(t):
            return torch.empty(n, ld, dtype=dtype, device="cuda")[:, :cols].copy_(t)
        xs, dys, dx = rows_of(x), rows_of(dy), rows_of(x)
        size = L.signmuon_layer_norm_backward_workspace_bytes(cols, rows)
        ws, kept = workspace(size)
        dw, db = torch.zeros(m, cols + 8, dtype=dtype, device="cuda"), torch.zeros(m, cols + 8, dtype=dtype, device="cuda")
        L.signmuon_layer_norm_backward(cols, rows, code, dys.data_ptr(), ld, xs.data_ptr(), ld, code, w.data_ptr(),
                                       stat.data_ptr(), stat.data_ptr(), dx.data_ptr(), ld,
                                       [dw[i].data_ptr() for i in range(m)], [db[i].data_ptr() for i in range(m)],
                                       ws.data_ptr(), size, stream)
        assert kept()
        for i in range(m):
            # Each sum is of at most n terms, and a rounding.
            part = dy[rows[i]:rows[i + 1]].double()
            e = (n + 8) * U * part.abs().sum(0)
            assert ((db[i, :cols].double() - part.sum(0)).abs() <= e + half(dtype) * (part.sum(0).abs() + e)).all()
    ids = torch.randint(0, 50, (n,), generator=g, device="cuda")
    size = L.signmuon_embedding_backward_workspace_bytes((50, cols), rows)
    ws, kept = workspace(size)
    table = torch.zeros(m, 50 * cols + 8, dtype=dtype, device="cuda")
    L.signmuon_embedding_backward((50, cols), rows, 1, ids.data_ptr(), code, dy.data_ptr(), cols, 1.0, 0, code,
                                  [table[i].data_ptr() for i in range(m)], ws.data_ptr(), size, stream)
    assert kept() and not table[:, 50 * cols:].any()
    top = min(cols, 3)
    size = L.signmuon_distill_workspace_bytes(n, top)
    ws, kept = workspace(size)
    loss, row, dz = torch.zeros(m, device="cuda"), torch.zeros(n, device="cuda"), torch.empty_like(x)
    top_ids = torch.randint(0, cols, (n, top), generator=g, device="cuda")
    L.signmuon_distill_loss(cols, rows, code, x.data_ptr(), cols, top, 1, top_ids.data_ptr(), 0, stat.repeat(top).data_ptr(),
                            1.0, 1.0, loss.data_ptr(), row.data_ptr(), dz.data_ptr(), cols, ws.data_ptr(), size, stream)
    assert kept()


@pytest.mark.gpu
def test_autograd_sees_what_is_written(cuda_lib):
    """A tensor that a backward pass has saved and a call then writes to fails
    that pass; tensors of inference mode, which have no versions, are written
    to all the same."""
    x = torch.randn(8, 16, device="cuda")
    w, stat, ids = torch.ones(16, device="cuda"), torch.ones(8, device="cuda"), torch.arange(8, device="cuda")
    calls = [
        lambda out: layers.embedding_forward(x, ids, out=out),
        lambda out: layers.embedding_backward(ids, x, 8, out=[out]),
        lambda out: layers.embedding_backward(ids, x, 8, out=[out], accumulate=True),
        lambda out: layers.layer_norm_forward(x, w, out=out),
        lambda out: layers.layer_norm_backward(x, x, w, stat, stat, out=out),
        lambda out: layers.distill_loss_and_grad(x, ids[:, None], stat[:, None], out=out),
    ]
    for call in calls:
        leaf = torch.randn(8, 16, device="cuda", requires_grad=True)
        saved = leaf.exp()
        with torch.no_grad():
            call(saved)
        assert saved._version == 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()
        with torch.inference_mode():
            plain = torch.zeros(8, 16, device="cuda")
            call(plain)
        call(plain)
        assert plain.any()
    assert x._version == 0 and w._version == 0


def test_overlap_of_row_tensors(lib):
    """Against the sets of bytes themselves, over views of one buffer."""
    overlap = layers._load().overlap
    buf = torch.zeros(400)
    where = torch.arange(400)
    views = [(off, n, cols, ld) for off in (0, 1, 5, 17, 40, 83, 200) for n in (1, 2, 5) for cols in (1, 4, 12)
             for ld in (12, 16, 21) if off + (n - 1) * ld + cols <= 400]
    tensors = [buf[off:].as_strided((n, cols), (ld, 1)) for off, n, cols, ld in views]
    bytes_of = [set(where[off:].as_strided((n, cols), (ld, 1)).flatten().tolist()) for off, n, cols, ld in views]
    for (va, a, sa) in zip(views, tensors, bytes_of):
        for (vb, b, sb) in zip(views, tensors, bytes_of):
            known = va[3] == vb[3] or a.is_contiguous() or b.is_contiguous() or va[1] == 1 or vb[1] == 1
            if known:
                assert overlap(a, b) == bool(sa & sb), (va, vb)
            else:
                assert not overlap(a, b) or sa & sb
    assert not overlap(buf[:0], buf) and not overlap(buf, torch.zeros(400))


@pytest.mark.gpu
def test_rows_that_overlap_are_refused(cuda_lib):
    """Outputs whose rows lie partly over an input's rows; columns of one buffer
    that do not are taken."""
    buf = torch.randn(8, 40, device="cuda")
    w, stat, ids = torch.ones(16, device="cuda"), torch.ones(8, device="cuda"), torch.arange(8, device="cuda")
    x, over, beside = buf[:, :16], buf[:, 8:24], buf[:, 16:32]
    calls = [
        lambda out: layers.embedding_forward(x, ids, out=out),
        lambda out: layers.layer_norm_forward(x, w, out=out)[0],
        lambda out: layers.layer_norm_backward(x, x.clone(), w, stat, stat, out=out)[0],
        lambda out: layers.layer_norm_backward(x.clone(), x, w, stat, stat, out=out)[0],
        lambda out: layers.distill_loss_and_grad(x, ids[:, None], stat[:, None], out=out)[2],
    ]
    for call in calls:
        kept = buf.clone()
        for bad in (over, buf[:, 1:17], torch.as_strided(buf, (8, 16), (40, 1), 5)):
            with pytest.raises(ValueError, match="overlap"):
                call(bad)
        assert torch.equal(buf, kept)
        want = call(torch.empty(8, 16, device="cuda"))
        assert torch.equal(call(beside), want) and torch.equal(buf[:, :16], kept[:, :16]) and torch.equal(buf[:, 32:], kept[:, 32:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_readme_training_example(cuda_lib, dtype):
    """The README's passes over a tied table, run as they stand there, against
    autograd on each worker's rows."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        code, = (c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "embedding_backward" in c)
    workers, rows, vocab, d, top = 8, 128, 160, 64, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)
    table, w, b = normal(vocab, d, std=0.5), normal(d, std=0.1, mean=1.0), normal(d, std=0.1)
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    top_ids = torch.rand(rows, vocab, generator=g, device="cuda").topk(top, dim=1).indices
    top_logits = torch.randn(rows, top, generator=g, device="cuda")
    here = dict(table=table, w=w, b=b, ids=ids, top_ids=top_ids, top_logits=top_logits)
    exec(code, here)
    t, per = 2.0, rows // workers
    # Six roundings to the type on the way, each amplified by the sums in between by at most sqrt(d).
    tol = 6 * d ** 0.5 * half(dtype) + 1e-5
    for m in range(workers):
        at = slice(m * per, (m + 1) * per)
        T, W, B = (q.double().requires_grad_() for q in (table, w, b))
        Y = torch.nn.functional.layer_norm(T[ids[at]], (d,), W, B, 1e-5)
        logp = torch.log_softmax(top_logits[at].double() / t, 1)
        logq = torch.log_softmax(Y @ T.t() / t, 1).gather(1, top_ids[at])
        ref = (logp.exp() * (logp - logq)).sum() * t * t / per
        ref.backward()
        assert abs(here["loss"][m].item() - ref.item()) <= tol * abs(ref.item())
        for got, want in ((here["d_table"][m], T.grad), (here["dw"][m], W.grad), (here["db"][m], B.grad)):
            assert (got.double() - want).norm() <= tol * want.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,top_dtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("shares,vocab,top,kind,extra", DISTILL)
@pytest.mark.parametrize("temperature", [0.5, 4.0])
def test_distill_gradient_in_place_and_at_other_addresses(cuda_lib, dtype, top_dtype, shares, vocab, top, kind, extra,
                                                          temperature):
    """The gradient over the logits, and into rows that lie differently within
    16 bytes, with losses: each within the bounds of the call that has a buffer
    of its own."""
    z, ids, u, splits = distill_inputs(shares, vocab, top, dtype, kind, seed=1, extra=extra, top_dtype=top_dtype,
                                       ids_dtype=torch.int64 if top % 2 else torch.int32)
    n, t = len(shares), temperature
    ref = distill_reference(z, ids, u, splits, t)
    bounds = distill_bounds(z, u, splits, t, top, ref)
    for out in (padded(torch.zeros(z.shape, dtype=dtype, device="cuda"), 3, offset=1), z):
        got = layers.distill_loss_and_grad(z, ids, u, n, splits, temperature=t, out=out)
        assert got[2] is out
        check_result(got, ref, bounds)
        dead = ~ref[5]
        assert not got[1][dead].any() and not out[dead].any()


def norm_reference(x, w, b, eps):
    """y, mean, 1 / std and what each may be off, as in test_layer_norm_forward."""
    X, W = x.double(), w.double()
    mu = X.mean(1)
    r = ((X - mu[:, None]).square().mean(1) + eps).rsqrt()
    depth = 64 + x.shape[1] / 512
    e_mu = depth * U * X.abs().mean(1) + U * mu.abs()
    e_r = (depth + 8) * U + 2 * e_mu * r
    xh = (X - mu[:, None]) * r[:, None]
    e_xh = (e_mu * r)[:, None] + (e_r[:, None] + 3 * U) * xh.abs()
    e = e_xh * W.abs() + 2 * U * ((xh * W).abs() + b.double().abs())
    y = xh * W + b.double()
    return (y, mu, r), (e + half(x.dtype) * (y.abs() + e), e_mu, e_r * r)


def norm_grad_reference(dy, x, w, mean, rstd, splits):
    """dx, dw, db and what they may be off, as in test_layer_norm_backward."""
    r, D = rstd.double()[:, None], dy.double()
    xh = (x.double() - mean.double()[:, None]) * r
    gy = D * w.double()
    s1, s2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    dx = r * (gy - s1 - xh * s2)
    depth = 64 + x.shape[1] / 512
    e1 = (depth + 2) * U * gy.abs().mean(1, keepdim=True)
    e2 = (depth + 6) * U * (gy * xh).abs().mean(1, keepdim=True)
    e = r * (U * gy.abs() + e1 + xh.abs() * e2 + 4 * U * (gy.abs() + s1.abs() + (xh * s2).abs()) + 2 * U * xh.abs() * s2.abs())
    out = [(dx, e + half(x.dtype) * (dx.abs() + e))]
    for terms in (D * xh, D):
        for a, b in zip(splits, splits[1:]):
            ref, e = terms[a:b].sum(0), (b - a + 12) * U * terms[a:b].abs().sum(0)
            out.append((ref, e + half(w.dtype) * (ref.abs() + e)))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [5, 8, 13, 16, 30, 60, 125, 256, 500, 512, 768, 1000, 1024, 1500, 1536, 2048, 2100, 4096, 5001, 8192,
                                  8200, 12288, 12300])
@pytest.mark.parametrize("offsets", [(1, 1, 1), (0, 1, 0), (3, 3, 2)])
def test_layer_norm_off_16_bytes(cuda_lib, dtype, cols, offsets):
    """Every division of a row among threads, element by element: x, dy and the
    outputs some elements past 16 bytes, and not all alike; what lies around the
    outputs' rows stays."""
    shares = [5, 0, 18] if cols < 2000 else [3, 4]
    splits = [sum(shares[:i]) for i in range(len(shares) + 1)]
    n, m = splits[-1], len(shares)
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    def lay(t, i):
        return padded(t, offsets[i] + 2, offset=offsets[i])
    x, dy = lay(normal(n, cols, std=2.0, mean=1.0), 0), lay(normal(n, cols), 1)
    w, b = normal(cols, std=0.2, mean=1.0), normal(cols)
    y = lay(torch.zeros(n, cols, dtype=dtype, device="cuda"), 2)
    got = layers.layer_norm_forward(x, w, b, out=y)
    for a, ref, e in zip(got, *norm_reference(x, w, b, 1e-5)):
        assert ((a.double() - ref).abs() <= e).all()
    dx = lay(torch.zeros(n, cols, dtype=dtype, device="cuda"), 2)
    ref = norm_grad_reference(dy, x, w, got[1], got[2], splits)
    got = layers.layer_norm_backward(dy, x, w, got[1], got[2], m, splits, out=dx)
    for a, (r, e) in zip((got[0], *got[1], *got[2]), ref):
        assert ((a.double() - r).abs() <= e).all()
    for out in (y, dx):
        assert out._base.isnan().sum() == n * (offsets[2] + 2)


@pytest.mark.gpu
def test_rows_beyond_two_to_the_31_elements(cuda_lib):
    """The last rows of buffers of more than 2^31 elements, against calls on
    those rows alone."""
    n, cols, last = 540000, 4096, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    assert (n - last) * cols > 1 << 31
    table = torch.randn(n, cols, generator=g, device="cuda", dtype=BF16)
    ids = torch.randperm(n, generator=g, device="cuda")
    y = layers.embedding_forward(table, ids)
    assert torch.equal(y[-last:], table[ids[-last:]]) and torch.equal(y[:last], table[ids[:last]])
    grad, = layers.embedding_backward(ids, y, n)          # every id once: the table again
    assert torch.equal(grad, table)
    del grad, y
    w = torch.randn(cols, generator=g, device="cuda")
    y, mean, rstd = layers.layer_norm_forward(table, w, out=table)
    assert y is table
    x = torch.randn(n, cols, generator=g, device="cuda", dtype=BF16)
    y, mean, rstd = layers.layer_norm_forward(x, w)
    for a, b in zip((y, mean, rstd), layers.layer_norm_forward(x[-last:], w)):
        assert torch.equal(a[-last:], b)
    del y
    dx, dw, db = layers.layer_norm_backward(table, x, w, mean, rstd, 2, [0, n - last, n])
    few = layers.layer_norm_backward(table[-last:], x[-last:], w, mean[-last:], rstd[-last:])
    assert torch.equal(dx[-last:], few[0])
    D = table[-last:].double()
    xh = (x[-last:].double() - mean[-last:, None].double()) * rstd[-last:, None].double()
    for got, terms in ((dw[1], D * xh), (db[1], D)):
        # Sums of `last` terms, in whatever blocks.
        assert ((got.double() - terms.sum(0)).abs() <= (last + 16) * U * terms.abs().sum(0) + U * terms.sum(0).abs()).all()
    del table, dx, x, D, xh
    n, vocab = 44000, 50008
    assert (n - last) * vocab > 1 << 31
    z = torch.randn(n, vocab, generator=g, device="cuda", dtype=BF16)
    z[-last // 2] = -1e30                                  # one that fp64 has
    top_ids, u = torch.randint(0, vocab, (n, 5), generator=g, device="cuda"), torch.randn(n, 5, generator=g, device="cuda")
    few = layers.distill_loss_and_grad(z[-last:].contiguous(), top_ids[-last:].contiguous(), u[-last:].contiguous())
    _, row, dz = layers.distill_loss_and_grad(z, top_ids, u, 2, [0, n - last, n], out=z)
    assert ((row[-last:] - few[1]).abs() <= 128 * U * (1 + few[1].abs())).all()
    # The same rows by other numbers of threads: sums of at most 128 terms in fp32, and bf16's roundings.
    a, b = dz[-last:].double(), few[2].double()
    assert ((a - b).abs() <= (128 * U + 2.0 ** -7) * b.abs() + 2.0 ** -126).all()
