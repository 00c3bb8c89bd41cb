"""Verification of drafted tokens against its 64-bit form: the same tokens."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import draft
from tests import mx4_ref, step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _exact(v, dtype):
    if dtype == "bf16":
        return mx4_ref.bf16_to_f64(mx4_ref.f64_to_bf16_bits(v))
    return v.astype(np.float32).astype(np.float64)


def _dev(v, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


def _case(B, D, V, dtype="f32", probs=None, seed=0, noise=0.5):
    """Logits, drafts a nearby distribution gave, random numbers, ragged lengths and
    temperatures, some 0."""
    rng = np.random.default_rng(seed + 31 * B + 7 * D + V)
    logits = _exact(2.5 * rng.standard_normal((B, D + 1, V)), dtype)
    tau = np.where(rng.random(B) < 0.25, 0.0, rng.uniform(0.4, 1.6, B)).astype(np.float32)
    guess = (logits[:, :D] + noise * rng.standard_normal((B, D, V))) \
        / np.where(tau > 0, tau, 1.0)[:, None, None]
    g = -np.log(-np.log(rng.random((B, D, V))))
    drafts = (guess + g * (tau > 0)[:, None, None]).argmax(-1) if D else np.zeros((B, 0), int)
    q = None
    if probs is not None:
        q = np.exp(guess - guess.max(-1, keepdims=True)) if D else np.zeros((B, 0, V))
        q = _exact(q / np.maximum(q.sum(-1, keepdims=True), 1e-300), probs)
    return {"logits": logits, "drafts": drafts, "uniforms": rng.random((B, D + 1)).astype(np.float32),
            "probs": q, "lengths": rng.integers(0, D + 1, B).astype(np.int32), "tau": tau}


def _call(c, dtype="f32", probs=None, wide=False, **kw):
    d = torch.from_numpy(np.ascontiguousarray(c["drafts"])).cuda()
    opt = {}
    if c["probs"] is not None:
        opt["draft_probs"] = _dev(c["probs"], TYPES[probs])
    if c["lengths"] is not None:
        opt["lengths"] = torch.from_numpy(c["lengths"]).cuda()
    if c["tau"] is not None:
        opt["temperature"] = _dev(c["tau"])
    opt.update(kw)
    return draft.draft_verify(opt.pop("logits", None) if "logits" in opt else
                              _dev(c["logits"], TYPES[dtype]), d if wide else d.to(torch.int32),
                              _dev(c["uniforms"]), **opt)


def _check(c, dtype="f32", probs=None, **kw):
    tokens, accepted = _call(c, dtype, probs, **kw)
    want, n = ref.verify(c["logits"], c["drafts"], c["uniforms"], c["probs"], c["lengths"], c["tau"])
    assert np.array_equal(accepted.cpu().numpy(), n)
    assert np.array_equal(tokens.cpu().numpy(), want)
    return n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("probs", [None, "f32", "bf16"])
@pytest.mark.parametrize("B,D,V", [(1, 0, 1), (1, 4, 32003), (3, 1, 7), (2, 3, 2048), (5, 7, 2049),
                                   (64, 2, 1000), (4, 15, 8200), (9, 0, 5000), (2, 70, 333),
                                   (33, 5, 65)])
def test_verify(B, D, V, probs, dtype):
    c = _case(B, D, V, dtype, probs)
    _check(c, dtype, probs)
    _check({**c, "lengths": None, "tau": None}, dtype, probs, wide=True)


def test_verify_long_rows_and_many_chunks():
    c = _case(2, 2, 151937, "f32", "f32")
    _check(c, "f32", "f32")
    c = _case(1, 1, 1 << 20, "bf16", None)
    _check(c, "bf16")


@pytest.mark.parametrize("probs", [None, "f32"])
def test_every_count_of_accepted_tokens_occurs(probs):
    counts = set()
    for seed in range(6):
        counts |= set(_check(_case(24, 6, 50, "f32", probs, seed, 0.3), "f32", probs))
    assert counts == set(range(7))


@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan])
@pytest.mark.parametrize("probs", [None, "f32"])
def test_random_numbers_at_and_past_their_ends(u, probs):
    """0 draws the first word of positive weight, 1 and above the last."""
    c = _case(12, 3, 4100, "f32", probs, 5)
    c["logits"][:, :, :40] = -np.inf
    c["logits"][:, :, -30:] = -np.inf
    c["drafts"] = np.clip(c["drafts"], 40, 4069)
    c["uniforms"][:, -1] = u
    _check(c, "f32", probs)
    c["uniforms"][:] = u
    _check(c, "f32", probs)


def test_rows_without_a_distribution():
    """NaN, +inf, all -inf: refused there, and -1 behind the accepted."""
    for probs in (None, "f32"):
        c = _case(8, 4, 600, "f32", probs, 3)
        c["lengths"] = None
        c["tau"] = np.array([0, 0, 0, 1, 1, 1, 0.7, 0], np.float32)
        best = c["logits"].argmax(-1)
        c["drafts"] = best[:, :4].copy()
        c["uniforms"][:, :4] = 0.0
        if probs is not None:
            c["probs"][:] = 1e-3
        for b, (row, bad) in enumerate([(2, np.nan), (0, np.inf), (4, None), (1, np.nan), (4, np.inf),
                                        (3, None), (4, np.nan)]):
            c["logits"][b, row, 17 if bad is not None else slice(None)] = \
                bad if bad is not None else -np.inf
        n = _check(c, "f32", probs)
        assert list(n) == [2, 0, 4, 1, 4, 3, 4, 4]


def test_masked_words():
    """-inf logits: never drawn; a draft that is one is refused."""
    for probs in (None, "bf16"):
        c = _case(16, 3, 3000, "f32", probs, 9)
        rng = np.random.default_rng(2)
        c["logits"][rng.random(c["logits"].shape) < 0.9] = -np.inf
        c["logits"][:, :, 11] = 0.0
        _check(c, "f32", probs)


def test_one_word_left():
    """Behind a refused draft with all the probability, the target's own is drawn."""
    c = _case(4, 1, 500, "f32", None, 1)
    c["logits"][:] = -np.inf
    c["logits"][:, :, 77] = 1.0
    c["drafts"][:] = 77
    c["uniforms"][:, 0] = 1.0                   # refused although p = 1
    c["tau"][:], c["lengths"] = 1.0, None
    tokens, n = _call(c)
    assert n.tolist() == [0] * 4 and tokens[:, 0].tolist() == [77] * 4
    _check(c)


def test_drafters_distribution_equal_to_the_targets_or_above_it():
    """max(0, p - q) is 0 everywhere: the target's own is drawn."""
    c = _case(6, 2, 900, "f32", "f32", 4)
    c["probs"][:] = 1.0
    c["lengths"] = None
    c["uniforms"][:, 0] = 0.9
    _check(c, "f32", "f32")


@pytest.mark.parametrize("probs", [None, "f32"])
def test_drafts_outside_the_vocabulary(probs):
    c = _case(6, 3, 100, "f32", probs, 8)
    c["lengths"] = None
    c["drafts"] = c["drafts"].astype(np.int64)
    c["drafts"][0, 0], c["drafts"][1, 1], c["drafts"][2, 0] = -1, 100, 2 ** 31 - 1
    _check(c, "f32", probs)
    c["drafts"][3, 0], c["drafts"][4, 0], c["drafts"][5, 2] = 2 ** 40, -2 ** 50, 2 ** 32 + 3
    _check(c, "f32", probs, wide=True)


def test_lengths_outside_their_range():
    c = _case(4, 3, 64, "f32", None, 2)
    c["lengths"] = np.array([-5, 99, 3, 0], np.int32)
    _check(c)


def test_rows_behind_a_sequences_last_are_not_read():
    """NaN there changes nothing."""
    c = _case(6, 5, 700, "f32", "f32", 6)
    a = _call(c, "f32", "f32")
    for b in range(6):
        c["logits"][b, c["lengths"][b] + 1:] = np.nan
    b = _call(c, "f32", "f32")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tau", [np.inf, 1e30, 1e-3, 1e-30, 1e-45, -1.0, np.nan])
def test_temperatures_far_out(tau):
    c = _case(5, 2, 300, "f32", None, 7)
    c["tau"] = np.full(5, tau, np.float32)
    _check(c)


@pytest.mark.parametrize("top", [9.0, 90.0])
def test_ties_of_the_largest_logit_go_to_the_lowest(top):
    """9 lies below some normal draws of 20000, 90 above all."""
    c = _case(6, 2, 20000, "bf16", None, 3)
    c["tau"][:], c["lengths"] = 0.0, None
    c["logits"][:, :, [19999, 8191, 8192, 300, 301]] = top
    c["logits"][3:, :, 5] = top
    c["drafts"][:, 0] = [300, 301, 300, 5, 300, 5]
    n = _check(c, "bf16")
    if top == 90.0:
        assert list(n > 0) == [True, False, True, True, False, True]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_unaligned_rows(dtype):
    """Every place of a row against the 16-byte boundaries, rows and sequences apart, the
    words beside them NaN; the drafter's probabilities too."""
    c = _case(3, 2, 4097, dtype, dtype, 11)
    want = _call(c, dtype, dtype)
    size = 4 if dtype == "f32" else 2
    for off in range(16 // size):
        for gap in (0, 1, 6):
            full = torch.full((3, 4, 4097 + off + gap), float("nan"), device="cuda",
                              dtype=TYPES[dtype])
            view = full[:, 1:, off:off + 4097]
            view[:] = _dev(c["logits"], TYPES[dtype])
            q = torch.full((2, 3, 4097 + off + gap), float("nan"), device="cuda",
                           dtype=TYPES[dtype]).transpose(0, 1)[:, :, off:off + 4097]
            q[:] = _dev(c["probs"], TYPES[dtype])
            ok = q.stride(1) >= 4097
            got = _call(c, dtype, dtype, logits=view, draft_probs=q if ok else q.contiguous())
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_given_outputs_and_workspace():
    c = _case(5, 4, 9000, "f32", "f32", 12)
    want = _call(c, "f32", "f32")
    need = draft.draft_workspace_bytes(5, 4, 9000)
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    t = torch.full((7, 5), 9, dtype=torch.int32, device="cuda")
    a = torch.full((7,), 9, dtype=torch.int32, device="cuda")
    got = _call(c, "f32", "f32", tokens=t[1:6], accepted=a[1:6], workspace=ws[:need])
    assert torch.equal(t[1:6], want[0]) and torch.equal(a[1:6], want[1])
    assert got[0].data_ptr() == t[1:6].data_ptr()
    assert bool((t[[0, 6]] == 9).all()) and bool((a[[0, 6]] == 9).all())
    assert bool((ws[need:] == 255).all())


def test_tokens_follow_the_targets_distribution():
    """20000 sequences that share one target: the first token's frequencies lie within
    six standard deviations of the target's probabilities."""
    B, V = 20000, 6
    rng = np.random.default_rng(1)
    target, guess = rng.standard_normal(V), rng.dirichlet(np.ones(V))
    p = np.exp(target) / np.exp(target).sum()
    logits = _dev(target).expand(B, 2, V).contiguous()
    drafts = torch.from_numpy(rng.choice(V, size=(B, 1), p=guess).astype(np.int32)).cuda()
    q = _dev(guess).expand(B, 1, V).contiguous()
    u = _dev(rng.random((B, 2)).astype(np.float32))
    tokens, _ = draft.draft_verify(logits, drafts, u, draft_probs=q)
    f = np.bincount(tokens[:, 0].cpu().numpy(), minlength=V) / B
    assert np.all(np.abs(f - p) <= 6 * np.sqrt(p * (1 - p) / B))


def test_more_sequences_than_one_launch_axis_holds():
    """2^22 and some sequences by workgroups of 1024 threads: more than 2^32 work items."""
    P, V = 64, 5
    B = (1 << 22) + 2 * P
    rng = np.random.default_rng(4)
    logits, u = _dev(rng.standard_normal((P, 1, V))), _dev(rng.random((P, 1)))
    none = torch.empty(P, 0, dtype=torch.int32, device="cuda")
    want, _ = draft.draft_verify(logits, none, u)
    assert len(set(want.flatten().tolist())) == V
    tokens, accepted = draft.draft_verify(logits.repeat(B // P, 1, 1),
                                          none.new_empty((B, 0)), u.repeat(B // P, 1))
    assert torch.equal(tokens.view(-1, P), want.view(1, P).expand(B // P, P))
    assert bool((accepted == 0).all())
