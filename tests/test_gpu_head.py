"""GPU tests of the LM head's token log-probabilities (entropy, alternatives, gradient) and of
the distillation from a teacher's list, against the oracle in 64 bits.

Tolerances.  The inputs' products sum exactly in fp32 (make_head_case), so a logit is off by its
scaling alone (2^-23 relative, 3e-6 at |z| <= 20).  e^d is off by (2^-22 + |d|·2^-23) relative, a
tile's sums by 128 roundings of 2^-24; averaged over p (Σ p|d| <= 12 here) that is 1.2e-5 in log Σe:
LP_ATOL.  The entropy's Σ d·e has the same relative error on a mean of up to 12: ENT_ATOL.  A
distillation loss adds q's error (2^-22 and 2^-23·|log q|) on terms of up to 20: LOSS_ATOL.

dX, recomputed: dz is rounded to bf16 once (2^-8 relative); exp's and the fp32 sums' errors stay
below 2^-10 of Σ|dz·W|; the result is rounded to bf16.  From a saved forward, e^z is rounded to bf16
(2^-8) and serves as dz itself; rows whose dz is written out (an entropy gradient, Σc small against
Σ|c|, an lse outside [-20, 60]) round it a second time, and take log p from the rounded e^z, off by
2^-8, on a term g·p.  Element by element, with r = 1 or 2 roundings:
|err| <= (r·2^-8 + 2^-10)·(|dz|·|W|) + (r - 1)·2^-8·scale·(Σ|c| + |g|)·(p·|W|) + 2^-8·|dX|
(the second term covers Σc - p·Σc on the given tokens as well).
"""
import numpy as np
import pytest
import torch

import oracle as O
from synth import HeadCase, make_head_case
from tests.gpu_helpers import dev_bf16, host_f64

pytestmark = pytest.mark.gpu

LP_ATOL, ENT_ATOL, LOSS_ATOL = 2e-5, 2e-4, 1e-4

# rows, width, vocabulary, tokens, alternatives: one entry and one row, ragged tiles, a
# vocabulary below one tile, both sides of the few-rows kernel's 128 rows, the longest lists
SHAPES = [(1, 8, 8, 1, 1), (3, 200, 1000, 1, 5), (1, 72, 20000, 2, 32), (40, 1000, 5000, 1, 8), (128, 64, 264, 2, 32),
          (129, 72, 520, 3, 7), (300, 200, 1000, 1, 0), (513, 328, 4096, 8, 20), (260, 64, 40000, 128, 32)]


def up(inp, *names):
    return [torch.from_numpy(np.ascontiguousarray(inp[k])).cuda() for k in names]


def head(lib, inp, cls, **kw):
    return cls(lib.LoraWeight.bf16(dev_bf16(inp["W"])), **kw)


def check_dX(name, dX, ref, W, gsum, T, r=1):
    """gsum: Σ|c| + |g| per row; r: roundings of dz."""
    aw = np.abs(W)
    z = ref["z"]
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    bound = (r * 2.0 ** -8 + 2.0 ** -10) * (np.abs(ref["dz"]) @ aw) + 2.0 ** -8 * np.abs(ref["dX"]) + \
        (r - 1) * (2.0 ** -8 / T) * gsum[:, None] * (p @ aw) + 1e-30
    got = host_f64(dX)
    assert np.all(np.isfinite(got)), name
    worst = np.max(np.abs(got - ref["dX"]) / bound)
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound"


def close(name, got, ref, atol):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, name
    err = np.max(np.abs(got - ref)) if ref.size else 0.0
    assert err <= atol, f"{name}: {err:.3e}"


def check_logprobs(out, ref, k, shape=None):
    close("logprob", out.logprob, ref["logprob"].reshape(out.logprob.shape), LP_ATOL)
    close("entropy", out.entropy, ref["entropy"], ENT_ATOL)
    if k:
        assert np.array_equal(out.top_ids.cpu().numpy(), ref["top_ids"])
        close("top_logprob", out.top_logprob, ref["top_logprob"], LP_ATOL)


def grads(inp):
    return (np.abs(inp["dlogprob"]).sum(1) + np.abs(inp["dentropy"])).astype(np.float64)


@pytest.mark.parametrize("T", [1.0, 0.7])
@pytest.mark.parametrize("M,D,V,n,k", SHAPES)
def test_logprobs(lib, M, D, V, n, k, T):
    inp = make_head_case(HeadCase("lp", M, D, V, n, 100 + M + V))
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    ref = O.token_logprobs(X, W, inp["ids"], -100, T, k, inp["dlogprob"], inp["dentropy"])
    layer = head(lib, inp, lib.LoraTokenLogProbs, temperature=T)
    x = dev_bf16(inp["X"])
    ids, dlp, dent = up(inp, "ids", "dlogprob", "dentropy")
    out = layer.forward(x, ids, top_k=k)
    check_logprobs(out, ref, k)
    check_dX("recomputed", layer.backward(x, ids, out, dlp, dent), ref, W, grads(inp), T)
    out = layer.forward(x, ids, top_k=k, save=True)
    check_logprobs(out, ref, k)
    check_dX("saved", layer.backward(x, ids, out, dlp, dent), ref, W, grads(inp), T, 2)
    assert out.saved is None  # used up: a second backward recomputes
    check_dX("second", layer.backward(x, ids, out, dlp, dent), ref, W, grads(inp), T)
    sliced = head(lib, inp, lib.LoraTokenLogProbs, temperature=T, slice_=256)
    check_dX("sliced", sliced.backward(x, ids, out, dlp, dent), ref, W, grads(inp), T)
    assert layer.status() == lib.LORA_OK and sliced.status() == lib.LORA_OK


@pytest.mark.parametrize("what", ["dlogprob", "dentropy"])
def test_logprob_gradients_one_at_a_time(lib, what):
    inp = make_head_case(HeadCase("one", 200, 96, 1032, 2, 61))
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    ref = O.token_logprobs(X, W, inp["ids"], -100, 1.0, 0, **{what: inp[what]})
    layer = head(lib, inp, lib.LoraTokenLogProbs)
    x = dev_bf16(inp["X"])
    ids, g = up(inp, "ids", what)
    for save in (False, True):
        out = layer.forward(x, ids, save=save)
        check_dX(what, layer.backward(x, ids, out, **{what: g}), ref, W, grads(inp), 1.0, 2 if save else 1)
    out = layer.forward(x, ids)
    assert torch.count_nonzero(layer.backward(x, ids, out)) == 0  # no upstream gradient
    nothing = layer.forward(x, None, top_k=3, entropy=False)
    assert nothing.logprob is None and nothing.entropy is None
    assert torch.equal(nothing.lse, out.lse)


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("M,D,V,n", [(1, 8, 8, 1), (5, 200, 1000, 16), (128, 64, 264, 3), (129, 328, 4096, 8),
                                     (300, 72, 2056, 128), (514, 136, 1000, 33)])
def test_distillation(lib, M, D, V, n, T):
    inp = make_head_case(HeadCase("kd", M, D, V, n, 300 + M + V))
    inp["teacher"][M // 2] = -np.inf          # a row without mass
    inp["ids"][M // 3] = -100                 # and one without entries
    if n > 2:
        inp["teacher"][::2, 1] = -np.inf
        inp["ids"][::5, 2] = inp["ids"][::5, 0]  # an id twice
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    ref = O.distill(X, W, inp["ids"], inp["teacher"], -100, T, inp["dloss"])
    layer = head(lib, inp, lib.LoraDistill, temperature=T)
    x = dev_bf16(inp["X"])
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    gs = 2.0 * inp["dloss"].astype(np.float64)
    for save in (False, True):
        out = layer.forward(x, ids, t, save=save)
        close("loss", out.loss, ref["loss"], LOSS_ATOL)
        dX = layer.backward(x, ids, t, out, dl)
        check_dX(f"saved={save}", dX, ref, W, gs, T)
        zero = ref["q"].sum(1) == 0
        assert np.all(out.loss.cpu().numpy()[zero] == 0) and np.all(host_f64(dX)[zero] == 0)
    sliced = head(lib, inp, lib.LoraDistill, temperature=T, slice_=512)
    check_dX("sliced", sliced.backward(x, ids, t, out, dl), ref, W, gs, T)
    assert layer.status() == lib.LORA_OK


@pytest.mark.parametrize("kept", ["none", "one", "last", "every_third", "all_but_first_block"])
def test_distillation_of_few_rows_of_a_batch(lib, kept):
    """Rows without an entry cost nothing (they are left out of the products) and change nothing:
    prompts in front, padding behind, rows in between, a batch of nothing else."""
    M, D, V, n = 1100, 136, 1032, 5
    inp = make_head_case(HeadCase("few", M, D, V, n, 171, ignore_frac=0.05))
    keep = np.zeros(M, dtype=bool)
    keep[{"none": slice(0, 0), "one": slice(700, 701), "last": slice(M - 3, M), "every_third": slice(0, M, 3),
          "all_but_first_block": slice(256, M)}[kept]] = True
    inp["ids"][~keep] = -100
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    ref = O.distill(X, W, inp["ids"], inp["teacher"], -100, 1.0, inp["dloss"])
    layer = head(lib, inp, lib.LoraDistill)
    x = dev_bf16(inp["X"])
    x[torch.from_numpy(~keep).cuda()] = float("nan")  # whatever those rows hold
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    for save in (False, True, True):
        out = layer.forward(x, ids, t, save=save)
        close("loss", out.loss, ref["loss"], LOSS_ATOL)
        if save:
            dX = layer.backward(x, ids, t, out, dl, dX=torch.full_like(x, 7.0))
            check_dX(kept, dX, ref, W, 2.0 * inp["dloss"].astype(np.float64), 1.0)
            assert np.all(host_f64(dX)[ref["q"].sum(1) == 0] == 0)
    assert layer.status() == lib.LORA_OK


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("kind", ["zero_rows", "repeated", "ascending", "descending", "block_of_best"])
def test_alternatives_in_hard_orders(lib, M, kind):
    """Equal logits (padded rows, repeated entries), every tile better or worse than the last, all
    of the best in one tile; ids have to be the oracle's, smaller first among equal logits."""
    inp = make_head_case(HeadCase("hard", M, 64, 4104, 1, 71))
    V = 4104
    W = O.bf16_to_f64(inp["W"])
    X = O.bf16_to_f64(inp["X"])
    if kind == "zero_rows":
        X[::2] = 0
    elif kind == "repeated":
        W = W[np.arange(V) % 37]
    elif kind in ("ascending", "descending"):
        X[:] = 0
        X[:, 0] = 1
        W[:, 0] = np.arange(V) // 16 / 16.0 * (1 if kind == "ascending" else -1)
    else:
        X[:] = 0
        X[:, 0] = 1
        W[:, 0] = 0
        W[1500:1600, 0] = 1 + np.arange(100) / 128.0
    k = 32
    ref = O.token_logprobs(X, W, inp["ids"], -100, 1.0, k)
    to = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()  # noqa: E731  (exact: grid values)
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(to(W)))
    for kk in (1, 2, 5, 32):
        out = layer.forward(to(X), None, top_k=kk)
        assert np.array_equal(out.top_ids.cpu().numpy(), ref["top_ids"][:, :kk]), kk
        close("top_logprob", out.top_logprob, ref["top_logprob"][:, :kk], LP_ATOL)
    assert layer.status() == lib.LORA_OK


@pytest.mark.parametrize("kind", ["random", "ascending", "descending", "peaks", "equal"])
def test_alternatives_of_few_rows_over_long_ranges(lib, kind):
    """Several tiles a CTA, so that later chunks are kept or dropped by the bound of earlier ones; calls
    of other sizes in between on the same workspace."""
    V, M = 60008, 128
    inp = make_head_case(HeadCase("long", M, 16, V, 1, 72))
    W, X = O.bf16_to_f64(inp["W"]), O.bf16_to_f64(inp["X"])
    if kind != "random":
        X[:] = 0
        X[:, 0] = 1
        X[1::2, 0] = -1  # every other row the other way round
        v = np.arange(V)
        W[:] = 0
        W[:, 0] = {"ascending": v // 512 / 8.0, "descending": -(v // 512) / 8.0, "equal": 0.0 * v,
                   "peaks": np.where(v % 1009 == 1008, (v // 1009) / 4.0, -1.0)}[kind]
    ref = O.token_logprobs(X, W, inp["ids"], -100, 1.0, 32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).cuda()  # noqa: E731  (exact)
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(to(W)))
    for m in (128, 1, 33):
        for k in (32, 1, 5, 20, 2):
            out = layer.forward(to(X[:m]), None, top_k=k)
            assert np.array_equal(out.top_ids.cpu().numpy(), ref["top_ids"][:m, :k]), (m, k)
            close("top_logprob", out.top_logprob, ref["top_logprob"][:m, :k], LP_ATOL)
    assert layer.status() == lib.LORA_OK


@pytest.mark.parametrize("M", [4, 140])
def test_ids_out_of_range_ignored_and_twice(lib, M):
    inp = make_head_case(HeadCase("ids", M, 64, 520, 4, 81, ignore_frac=0.0))
    ids = inp["ids"]
    ids[0] = [519, 519, 0, -100]
    ids[1] = [520, 7, -1, -2147483648]
    ids[2] = [2147483647, 3, 3, 3]
    x = dev_bf16(inp["X"])
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    for ign in (-100, 7):  # an ignore_index that is an entry's id leaves that entry out
        ref = O.token_logprobs(X, W, ids, ign)
        layer = head(lib, inp, lib.LoraTokenLogProbs, ignore_index=ign)
        out = layer.forward(x, up(inp, "ids")[0])
        got = out.logprob.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref["logprob"]))
        ok = ~np.isnan(got)
        assert np.max(np.abs(got[ok] - ref["logprob"][ok])) <= LP_ATOL
        # the other rows' gradients stand whatever rows 1 and 2 hold
        dlp, = up(inp, "dlogprob")
        good = np.arange(M) > 2
        r = O.token_logprobs(X[good], W, ids[good], ign, 1.0, 0, inp["dlogprob"][good])
        for save in (False, True):
            o = layer.forward(x, up(inp, "ids")[0], save=save)
            dX = layer.backward(x, up(inp, "ids")[0], o, dlp)
            check_dX("rows", dX[3:], r, W, np.abs(inp["dlogprob"][good]).sum(1).astype(np.float64), 1.0,
                     2 if save else 1)
        assert layer.status() == lib.LORA_OK


@pytest.mark.parametrize("M", [6, 150])
def test_teachers_that_are_not_finite(lib, M):
    inp = make_head_case(HeadCase("nan", M, 64, 520, 4, 91, ignore_frac=0.0))
    t = inp["teacher"]
    t[0, 1] = np.nan
    t[1, 2] = np.inf
    t[2] = np.nan
    t[3, 0] = np.nan
    inp["ids"][3, 0] = -100          # a NaN in an ignored place says nothing
    t[4, 0] = -np.inf
    inp["ids"][4, 0] = 1000          # an id out of range without weight neither
    layer = head(lib, inp, lib.LoraDistill)
    x = dev_bf16(inp["X"])
    ids, tt = up(inp, "ids", "teacher")
    loss = layer.forward(x, ids, tt).loss.cpu().numpy()
    assert np.all(np.isnan(loss[:3])) and np.all(np.isfinite(loss[3:]))
    safe_t, safe_ids = t.copy(), inp["ids"].copy()
    safe_t[:3] = 0
    safe_t[3, 0] = 0
    safe_ids[4, 0] = 0
    ref = O.distill(O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"]), safe_ids, safe_t, -100)
    assert np.max(np.abs(loss[3:] - ref["loss"][3:])) <= LOSS_ATOL


@pytest.mark.parametrize("M", [7, 300])
def test_rows_that_are_not_finite_stay_alone(lib, M):
    """A row whose hidden state holds an infinity or a NaN gives NaN; its neighbours' results are
    those of a batch without it."""
    inp = make_head_case(HeadCase("inf", M, 64, 1000, 2, 95))
    x = dev_bf16(inp["X"])
    bad = x.clone()
    bad[1, 3] = float("inf")
    bad[4] = float("nan")
    layer = head(lib, inp, lib.LoraTokenLogProbs, ignore_index=-1000)
    ids = up(inp, "ids")[0].clamp(min=0)
    a, b = layer.forward(x, ids, top_k=4), layer.forward(bad, ids, top_k=4)
    rest = torch.tensor([i for i in range(M) if i not in (1, 4)], device="cuda")
    for name in ("logprob", "entropy", "lse", "top_ids", "top_logprob"):
        assert torch.equal(getattr(a, name)[rest], getattr(b, name)[rest]), name
    assert torch.isnan(b.lse[[1, 4]]).all() and torch.isnan(b.logprob[[1, 4]]).all()
    assert layer.status() == lib.LORA_OK


def test_saved_forward_over_the_range_of_logits(lib):
    """Rows whose logits a bf16 e^z cannot hold (around -64, around +130, tiles 64 below the rest),
    gradients that cancel (Σc = 0), rows without one and rows certain of their token, in one batch,
    from a saved forward: each as close as the bound for written-out rows."""
    M, D, V = 300, 64, 2056
    inp = make_head_case(HeadCase("range", M, D, V, 2, 161, ignore_frac=0.0))
    X, W = O.bf16_to_f64(inp["X"]), O.bf16_to_f64(inp["W"])
    ids, dlp = inp["ids"], inp["dlogprob"]
    W[:, 0] = 1.0
    W[:, 1] = np.where(np.arange(V) < 512, 0.0, -8.0)
    X[:, :2] = 0
    X[0::6, 0] = -64.0
    X[1::6, 0] = 130.0
    X[2::6, 1] = 8.0
    dlp[3::6] = [[1.0, -1.0]]
    dlp[4::6] = 0.0
    ids[5::6, 1] = ids[5::6, 0]
    W[ids[5::6, 0], 2] = 4.0
    X[5::6, 2] = 4.0
    inp["teacher"][:, 0] += 3.0
    to = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()  # noqa: E731  (exact: grid values)
    Wd, x = lib.LoraWeight.bf16(to(W)), to(X)
    lp, kd = lib.LoraTokenLogProbs(Wd), lib.LoraDistill(Wd)
    i, d, t, dl = up(inp, "ids", "dlogprob", "teacher", "dloss")
    ref = O.token_logprobs(X, W, ids, -100, 1.0, 0, dlp)
    out = lp.forward(x, i, save=True)
    close("logprob", out.logprob, ref["logprob"], 2e-4)  # 2^-24·|z| at |z| = 150 on top of LP_ATOL
    dX = lp.backward(x, i, out, d)
    check_dX("logprob", dX, ref, W, np.abs(dlp).sum(1).astype(np.float64), 1.0, 2)
    assert np.all(host_f64(dX)[4::6] == 0)
    ref = O.distill(X, W, ids, inp["teacher"], -100, 1.0, inp["dloss"])
    out = kd.forward(x, i, t, save=True)
    check_dX("distill", kd.backward(x, i, t, out, dl), ref, W, 2.0 * inp["dloss"].astype(np.float64), 1.0, 2)
    assert lp.status() == lib.LORA_OK and kd.status() == lib.LORA_OK


def test_empty_batch(lib):
    W = lib.LoraWeight.bf16(torch.zeros((256, 64), dtype=torch.bfloat16, device="cuda"))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    t = torch.empty((0, 3), device="cuda")
    lp, kd = lib.LoraTokenLogProbs(W), lib.LoraDistill(W)
    o = lp.forward(x, ids, top_k=2, save=True)
    assert o.logprob.shape == (0, 3) and o.top_ids.shape == (0, 2)
    assert lp.backward(x, ids, o, t, torch.empty(0, device="cuda")).shape == (0, 64)
    d = kd.forward(x, ids, t)
    assert kd.backward(x, ids, t, d, torch.empty(0, device="cuda")).shape == (0, 64)


def test_teacher_to_student(lib):
    """The operators as they are used together: a teacher's alternatives become the student's
    targets; a student that is the teacher has the loss of the list's missing mass."""
    ti = make_head_case(HeadCase("teacher", 260, 128, 2000, 1, 111))
    si = make_head_case(HeadCase("student", 260, 72, 2000, 1, 112))
    teacher, student = head(lib, ti, lib.LoraTokenLogProbs), head(lib, si, lib.LoraDistill)
    xt, xs = dev_bf16(ti["X"]), dev_bf16(si["X"])
    top = teacher.forward(xt, None, top_k=16, entropy=False)
    out = student.forward(xs, top.top_ids, top.top_logprob, save=True)
    dl = torch.full((260,), 1.0 / 260, device="cuda")
    dX = student.backward(xs, top.top_ids, top.top_logprob, out, dl)
    rt = O.token_logprobs(O.bf16_to_f64(ti["X"]), O.bf16_to_f64(ti["W"]), ti["ids"], -100, 1.0, 16)
    Ws = O.bf16_to_f64(si["W"])
    ref = O.distill(O.bf16_to_f64(si["X"]), Ws, rt["top_ids"], rt["top_logprob"], -100, 1.0, np.full(260, 1 / 260))
    close("loss", out.loss, ref["loss"], LOSS_ATOL)
    check_dX("dX", dX, ref, Ws, np.full(260, 2 / 260), 1.0)
    same = head(lib, ti, lib.LoraDistill).forward(xt, top.top_ids, top.top_logprob)
    mass = np.exp(rt["top_logprob"]).sum(1)
    close("self", same.loss, -np.log(mass), LOSS_ATOL)


def test_gradient_against_differences(lib):
    """Directional differences of the operators themselves: steps of 1/16 in X change logits by
    about 0.03, so the central difference is off by its third-order term (1e-4 of a derivative of
    order 1) and by the fp32 losses (2e-5/0.125); dX by its bf16 roundings (2^-7 of Σ|dz|)."""
    inp = make_head_case(HeadCase("fd", 160, 256, 1000, 3, 121, ignore_frac=0.0))
    x = dev_bf16(inp["X"])
    ids, t, dlp, dent = up(inp, "ids", "teacher", "dlogprob", "dentropy")
    lp, kd = head(lib, inp, lib.LoraTokenLogProbs), head(lib, inp, lib.LoraDistill)
    g = torch.Generator().manual_seed(3)
    for _ in range(3):
        step = (torch.randint(0, 2, x.shape, generator=g) * 2 - 1).to(torch.bfloat16).cuda() / 16
        step[torch.rand(x.shape, generator=g).cuda() < 0.9] = 0

        def f(xx):
            o = lp.forward(xx, ids)
            return (o.logprob * dlp).sum(1) + o.entropy * dent + kd.forward(xx, ids, t).loss

        diff = (f(x + step) - f(x - step)).double() / 2
        o = lp.forward(x, ids, save=True)
        d = kd.forward(x, ids, t, save=True)
        dX = lp.backward(x, ids, o, dlp, dent).double() + \
            kd.backward(x, ids, t, d, torch.ones(160, device="cuda")).double()
        want = (dX * step.double()).sum(1)
        scale = (dlp.abs().sum(1) + dent.abs() + 1).double()
        assert float(((diff - want).abs() / scale).max()) < 2e-2 * 0.5


def test_same_bits_every_time_and_rows_behind_stay(lib):
    inp = make_head_case(HeadCase("bits", 400, 128, 3000, 2, 131))
    x = dev_bf16(inp["X"])
    ids, dlp, dent = up(inp, "ids", "dlogprob", "dentropy")
    W = lib.LoraWeight.bf16(dev_bf16(inp["W"]))
    layer = lib.LoraTokenLogProbs(W)
    for M in (400, 100):
        runs = []
        for _ in range(3):
            o = layer.forward(x[:M], ids[:M], top_k=9, save=True)
            runs.append((o.logprob, o.entropy, o.lse, o.top_ids, o.top_logprob,
                         layer.backward(x[:M], ids[:M], o, dlp[:M], dent[:M])))
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
    # outputs and rows behind the batch's last are left alone
    M, k = 136, 8
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    lp, ent, lse, tl, ti = f(200, 2), f(200), f(200), f(200, k), torch.full((200, k), 7, dtype=torch.int32, device="cuda")
    dX = torch.full((200, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(max(lib.head_fwd_workspace_bytes(M, 128, 3000, 2, k),
                         lib.head_bwd_workspace_bytes(M, 128, 3000, 2, 512)), dtype=torch.uint8, device="cuda")
    for m in (M, 24):
        lib.lora_logprob_fwd(x, m, W, ids, 2, -100, 1.0, k, lp, ent, lse, ti, tl, None, ws)
        lib.lora_logprob_bwd(x, m, W, ids, 2, -100, 1.0, lse, ent, dlp, dent, None, dX, ws)
        for t in (lp, ent, lse, tl, ti, dX):
            assert torch.all(t[M:] == 7)
    assert lib.lora_device_status(ws) == lib.LORA_OK


def test_graphs_and_streams(lib):
    """Two captured graphs of one layer, replayed with new data after an ordinary call, and calls
    on two streams at once, give the bits of ordinary calls."""
    inp = make_head_case(HeadCase("graph", 300, 128, 3000, 4, 141))
    x, x2 = dev_bf16(inp["X"]), dev_bf16(inp["X"]).flip(0).contiguous()
    ids, t, dl, dlp, dent = up(inp, "ids", "teacher", "dloss", "dlogprob", "dentropy")
    lp, kd = head(lib, inp, lib.LoraTokenLogProbs), head(lib, inp, lib.LoraDistill)

    def step(xx):
        o = lp.forward(xx, ids, top_k=5, save=True)
        d = kd.forward(xx, ids, t, save=True)
        few = lp.forward(xx[:16], ids[:16], top_k=5)
        return [o.logprob, o.entropy, o.top_ids, d.loss, lp.backward(xx, ids, o, dlp, dent),
                kd.backward(xx, ids, t, d, dl), few.logprob, few.top_ids]

    want, want2 = step(x), step(x2)
    torch.cuda.synchronize()
    buf = x.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(buf)
        graphs.append((g, got))
    for data, ref in ((x2, want2), (x, want)):
        buf.copy_(data)
        for g, got in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(3):
        for s, data in ((s1, x), (s2, x2)):
            with torch.cuda.stream(s):
                res.append((step(data), want if data is x else want2))
    o1 = lp.forward(x, ids, top_k=5, stream=s1)
    o2 = lp.forward(x2, ids, top_k=5, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for got, ref in res:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert torch.equal(o1.logprob, want[0]) and torch.equal(o2.logprob, want2[0])
    assert lp.status() == lib.LORA_OK and kd.status() == lib.LORA_OK
    del graphs


@pytest.mark.parametrize("op", ["logprob", "distill"])
def test_captured_backward_of_an_ordinary_forward(lib, op):
    """Replays of a backward captured on its own all give the gradient, and the saved forward still
    serves an ordinary backward."""
    inp = make_head_case(HeadCase("graph_bwd", 300, 128, 3000, 4, 143))
    x = dev_bf16(inp["X"])
    ids, t, dl, dlp, dent = up(inp, "ids", "teacher", "dloss", "dlogprob", "dentropy")
    layer = head(lib, inp, lib.LoraTokenLogProbs if op == "logprob" else lib.LoraDistill)

    def fwd(save):
        return layer.forward(x, ids, save=save) if op == "logprob" else layer.forward(x, ids, t, save=save)

    def bwd(o):
        return layer.backward(x, ids, o, dlp, dent) if op == "logprob" else layer.backward(x, ids, t, o, dl)

    saved_way, recomputed = bwd(fwd(True)), bwd(fwd(False))
    o = fwd(True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = bwd(o)
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, recomputed)
    assert torch.equal(bwd(o), saved_way) and o.saved is None
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, recomputed)
    del g


def test_saved_forward_of_another_stream(lib):
    """A backward on another stream than its forward's: the saved buffer is not handed out on the
    forward's stream before the backward has run."""
    inp = make_head_case(HeadCase("other_stream", 300, 128, 3000, 4, 144))
    x = dev_bf16(inp["X"])
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    kd = head(lib, inp, lib.LoraDistill)
    want = kd.backward(x, ids, t, kd.forward(x, ids, t, save=True), dl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = kd.forward(x, ids, t, save=True, stream=s)
    torch.cuda.synchronize()
    where, size = o.saved.data_ptr(), o.saved.numel()
    torch.cuda._sleep(200_000_000)  # about 0.1 s, before the backward in its stream
    got = kd.backward(x, ids, t, o, dl)
    with torch.cuda.stream(s):
        other = torch.empty(size, dtype=torch.uint8, device=x.device)
    assert other.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [40, 250, 900])
def test_rows_without_a_gradient_hold_anything(lib, M):
    """NaN hidden states in rows that have no entry (or no upstream gradient) reach neither their own
    nor another row's gradient, recomputed in one piece, in slices or from a saved forward."""
    inp = make_head_case(HeadCase("pad", M, 64, 1000, 3, 181))
    inp["ids"][::4] = -100
    inp["dlogprob"][::4] = 0
    off = (inp["ids"] == -100).all(1)
    inp["dlogprob"][off] = 0
    W = O.bf16_to_f64(inp["W"])
    lr = O.token_logprobs(O.bf16_to_f64(inp["X"]), W, inp["ids"], -100, 1.0, 0, inp["dlogprob"])
    kr = O.distill(O.bf16_to_f64(inp["X"]), W, inp["ids"], inp["teacher"], -100, 1.0, inp["dloss"])
    x = dev_bf16(inp["X"])
    x[torch.from_numpy(off).cuda()] = float("nan")
    ids, t, dl, dlp = up(inp, "ids", "teacher", "dloss", "dlogprob")
    for kw in ({}, {"slice_": 512}):
        lp, kd = head(lib, inp, lib.LoraTokenLogProbs, **kw), head(lib, inp, lib.LoraDistill, **kw)
        for save in (False, True):
            o, d = lp.forward(x, ids, save=save), kd.forward(x, ids, t, save=save)
            close("loss", d.loss, kr["loss"], LOSS_ATOL)
            check_dX("logprob", lp.backward(x, ids, o, dlp), lr, W, grads(inp), 1.0, 2 if save else 1)
            check_dX("distill", kd.backward(x, ids, t, d, dl), kr, W, 2.0 * inp["dloss"].astype(np.float64), 1.0)


def test_same_bits_of_compacted_rows(lib):
    """Distillation's rows find their places in any order; their results are the same bits."""
    inp = make_head_case(HeadCase("order", 3000, 64, 1000, 4, 191, ignore_frac=1.0))
    x = dev_bf16(inp["X"])
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    layer = head(lib, inp, lib.LoraDistill)
    runs = []
    for _ in range(4):
        o = layer.forward(x, ids, t, save=True)
        runs.append((o.loss, layer.backward(x, ids, t, o, dl)))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


def test_a_larger_workspace_keeps_the_status(lib):
    inp = make_head_case(HeadCase("status", 300, 64, 3000, 1, 151))
    x = dev_bf16(inp["X"])
    layer = head(lib, inp, lib.LoraTokenLogProbs)
    layer.forward(x[:2])
    (ws,) = layer._ws.values()
    ws[:4].view(torch.int32).fill_(1)  # as a kernel that gave up a wait leaves it
    layer.forward(x, top_k=4)
    assert layer._ws[next(iter(layer._ws))].numel() > ws.numel()
    assert layer.status() == lib.LORA_ERR_DEVICE_TIMEOUT and layer.status() == lib.LORA_OK


def test_two_threads_on_one_stream(lib):
    import threading

    inp = make_head_case(HeadCase("threads", 300, 128, 3000, 4, 201))
    x = dev_bf16(inp["X"])
    ids, t, dl = up(inp, "ids", "teacher", "dloss")
    layer = head(lib, inp, lib.LoraDistill)
    xs = [x, x.flip(0).contiguous()]
    want = [layer.forward(v, ids, t).loss for v in xs]
    got = [[], []]

    def work(i):
        for _ in range(50):
            o = layer.forward(xs[i], ids, t, save=True)
            got[i].append((o.loss, layer.backward(xs[i], ids, t, o, dl)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(loss, want[i]) and torch.equal(dX, got[i][0][1]) for loss, dX in got[i])


def test_layer_checks(lib):
    inp = make_head_case(HeadCase("chk", 8, 64, 256, 2, 151))
    lp, kd = head(lib, inp, lib.LoraTokenLogProbs), head(lib, inp, lib.LoraDistill)
    x = dev_bf16(inp["X"])
    ids, t, dlp = up(inp, "ids", "teacher", "dlogprob")
    out = lp.forward(x, ids[:, 0].contiguous())
    assert out.logprob.shape == (8,)
    o = lp.forward(x, ids, entropy=False)
    for call in (lambda: lp.forward(x.float(), ids), lambda: lp.forward(x.t(), ids), lambda: lp.forward(x[:, :32], ids),
                 lambda: lp.forward(x, ids.long()), lambda: lp.forward(x, ids[:4]), lambda: lp.forward(x, ids.cpu()),
                 lambda: lp.forward(x, ids[:, ::2]), lambda: lp.forward(x, ids, top_k=33),
                 lambda: lp.forward(x, ids, top_k=-1), lambda: lp.backward(x, ids, o, dlp[:, 0]),
                 lambda: lp.backward(x, ids, o, dlp.half()), lambda: lp.backward(x, None, o, dlp),
                 lambda: lp.backward(x, ids, o, dlp, torch.ones(8, device="cuda")),
                 lambda: lp.backward(x[:4], ids[:4], o, dlp[:4]),
                 lambda: lp.backward(x, ids, o, dlp, dX=torch.empty((8, 64), device="cuda")),
                 lambda: lp.backward(x, ids[:, 0].contiguous(), lp.forward(x, ids, save=True)),
                 lambda: kd.forward(x, ids[:, 0].contiguous(), t), lambda: kd.forward(x, ids, t[:, :1]),
                 lambda: kd.forward(x, ids, t.double()), lambda: kd.forward(x, torch.zeros((8, 129), dtype=torch.int32,
                                                                                       device="cuda"), t)):
        with pytest.raises(ValueError):
            call()


def test_offsets_past_32_bits(lib):
    """20000 rows over 128256 entries: the saved buffer has 2.6e9 elements and the rows go
    through several chunks; sampled rows against the oracle."""
    M, D, V, n = 20000, 64, 128256, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    W = (torch.randn((V, D), generator=g, device="cuda") * 4).round_().clamp_(-120, 120).div_(16).to(torch.bfloat16)
    x = (torch.randn((M, D), generator=g, device="cuda") * 8).round_().div_(8).to(torch.bfloat16)
    ids = torch.randint(0, V, (M, n), generator=g, device="cuda", dtype=torch.int32)
    dlp = torch.randn((M, n), generator=g, device="cuda")
    layer = lib.LoraTokenLogProbs(lib.LoraWeight.bf16(W))
    rows = np.array([0, 1, 255, 256, 7777, 16383, 16384, 16743, 16744, 19998, 19999])
    Wn = W.double().cpu().numpy()
    pick = torch.from_numpy(rows).cuda()
    ref = O.token_logprobs(x[pick].double().cpu().numpy(), Wn, ids[pick].cpu().numpy(), -100, 1.0, 8,
                           dlp[pick].cpu().numpy())
    for save in (True, False):
        out = layer.forward(x, ids, top_k=8, save=save)
        dX = layer.backward(x, ids, out, dlp)
        sub = lib.TokenLogProbs(out.logprob[pick], None, out.entropy[pick], out.top_ids[pick], out.top_logprob[pick])
        check_logprobs(sub, ref, 8)
        check_dX(f"save={save}", dX[pick], ref, Wn, np.abs(dlp[pick].cpu().numpy()).sum(1).astype(np.float64), 1.0,
                 2 if save else 1)
    assert layer.status() == lib.LORA_OK
