"""Verification of drafted tokens on the GPU against the plain float64 form: counts and tokens
must be equal, in a layer's verification step with the rollback on the device too."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_02_b200 as Q
import synth
from oracle import paged_oracle as P
from oracle import qsa_oracle as O
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

BAD_INDEX = 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_library()


def _verify(target, draft, tokens, u, n_drafts=None, pad=0, status=None):
    S, rows, V = target.shape
    dev = lambda x, dt: None if x is None else H.to_dev(np.asarray(x, dt))  # noqa: E731

    def spread(x):      # rows `pad` floats further apart than they are long
        if x is None:
            return None
        wide = torch.full((*x.shape[:2], V + pad), float("nan"), device="cuda")
        wide[..., :V] = dev(x, np.float32)
        return wide[..., :V]

    acc, nxt = (torch.full((S,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    Q.verify_drafts(spread(target), spread(draft), dev(tokens, np.int32), dev(u, np.float32), acc, nxt,
                    n_drafts=dev(n_drafts, np.int32), status=status)
    return list(zip(acc.tolist(), nxt.tolist()))


def _random(rng, S, K, V, sharp=2.0):
    x = rng.standard_normal((S, K + 1, V)) * sharp
    soft = lambda z: (lambda e: (e / e.sum(-1, keepdims=True)).astype(np.float32))(np.exp(z - z.max(-1, keepdims=True)))  # noqa: E731
    target, draft = soft(x), soft(x[:, :K] + rng.standard_normal((S, K, V)) * 0.6)
    g = rng.gumbel(size=(S, K, V))
    tokens = np.argmax(np.log(draft.astype(np.float64) + 1e-300) + g, -1).astype(np.int32) if K else np.zeros((S, 0), np.int32)
    return target, draft, tokens, rng.random((S, K + 1), np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 33, 257, 1000, 4096, 32000, 50257, 151936])
@pytest.mark.parametrize("K", [0, 1, 3, 8])
@pytest.mark.parametrize("drafter", [True, False])
def test_equal_to_the_plain_form(V, K, drafter):
    rng = np.random.default_rng(V * 10 + K)
    S = 3 if V > 40000 else 9
    target, draft, tokens, u = _random(rng, S, K, V)
    draft = draft if drafter else None
    want = [P.verify(target[i], None if draft is None else draft[i], tokens[i], u[i]) for i in range(S)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert _verify(target, draft, tokens, u, status=status) == want
    assert _verify(target, draft, tokens, u, pad=3) == want
    assert int(status) == 0


@pytest.mark.parametrize("K", [31, 32, 33, 64])
def test_long_drafts(K):
    rng = np.random.default_rng(K)
    target, draft, tokens, u = _random(rng, 12, K, 500)
    for i in range(12):         # from none to all accepted
        u[i, :K] *= 1e-3 if i % 3 == 0 else 1.0
        u[i, min(i * 6, K - 1)] = 0.999 if i % 2 else 0.0
    u[0, :K] = u[1, :K] = 0.0   # everything with a probability
    want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(12)]
    assert max(m for m, _ in want) == K and min(m for m, _ in want) < 32
    assert _verify(target, draft, tokens, u) == want
    want = [P.verify(target[i], None, tokens[i], u[i]) for i in range(12)]
    assert _verify(target, None, tokens, u) == want


def test_large_vocabulary_and_batch():
    rng = np.random.default_rng(1)
    target, draft, tokens, u = _random(rng, 2, 1, 1_000_003)
    assert _verify(target, draft, tokens, u) == [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(2)]
    target, draft, tokens, u = _random(rng, 700, 2, 500)
    assert _verify(target, draft, tokens, u) == [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(700)]


@pytest.mark.parametrize("V", [8, 64, 1024, 65536])
def test_exact_thresholds(V):
    """Equal probabilities 1/V: every partial sum is exact, so u = j/V draws token j."""
    js = sorted({0, 1, V // 3, V // 2, V - 2, V - 1})
    target = np.full((len(js), 1, V), 1.0 / V, np.float32)
    u = np.array([[j / V] for j in js], np.float32)
    assert _verify(target, None, np.zeros((len(js), 0), np.int32), u) == [(0, j) for j in js]
    below = np.nextafter(u, np.float32(-1.0)).astype(np.float32)
    assert _verify(target, None, np.zeros((len(js), 0), np.int32), below) == [(0, max(j - 1, 0)) for j in js]


def test_ctas_with_few_or_no_tokens_of_a_row():
    """Vocabularies that leave the last CTAs of a cluster little or nothing to read: they reach
    the exchange of the sums long before the others, launch after launch."""
    rng = np.random.default_rng(12)
    for S, V in ((1, 4097), (1, 4225), (5, 4096), (20, 2049), (40, 2111), (70, 1030)):
        target, draft, tokens, u = _random(rng, S, 2, V)
        want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(S)]
        dev = [H.to_dev(x) for x in (target, draft, tokens, u)]
        outs = [[torch.full((S,), -7, dtype=torch.int32, device="cuda") for _ in range(2)] for _ in range(40)]
        for o in outs:
            Q.verify_drafts(*dev, *o)
        for o in outs:
            assert list(zip(o[0].tolist(), o[1].tolist())) == want


def test_batches_of_any_size_give_a_sequence_the_same_token():
    """A sequence alone, and in batches that give it 16, 8, 4, 2 and 1 CTAs."""
    rng = np.random.default_rng(21)
    target, draft, tokens, u = _random(rng, 330, 1, 6001)
    want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(330)]
    for n in (1, 18, 70, 140, 290, 330):
        for at in sorted({0, (330 - n) // 2, 330 - n}):
            s = slice(at, at + n)
            assert _verify(target[s], draft[s], tokens[s], u[s]) == want[s]


def test_all_weight_on_one_token():
    V = 70001
    for at in (0, 1, 35000, V - 1):
        target = np.zeros((4, 1, V), np.float32)
        target[:, 0, at] = 0.3
        got = _verify(target, None, np.zeros((4, 0), np.int32), np.array([[0.0], [0.5], [1.0], [np.nan]]))
        assert got == [(0, at)] * 4


def test_random_numbers_at_and_outside_their_range():
    rng = np.random.default_rng(2)
    target, draft, tokens, u = _random(rng, 6, 2, 300)
    target[:, :, -20:] = 0.0
    u[:, -1] = [0.0, -1.0, np.nan, 1.0, 2.0, 1.0 - 2.0 ** -24]
    want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(6)]
    assert _verify(target, draft, tokens, u) == want
    u[:, 0] = [0.0, -1.0, np.nan, 1.0, 2.0, 1e-30]      # a NaN accepts nothing, a negative number anything p > 0
    want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(6)]
    assert _verify(target, draft, tokens, u) == want


@pytest.mark.parametrize("K", [1, 3, 40])
def test_negative_random_numbers_count_as_zero(K):
    """A draft whose token the target never gives is not accepted by a negative number either."""
    rng = np.random.default_rng(K)
    target, draft, tokens, u = _random(rng, 8, K, 90)
    at = [0, K - 1, K // 2, 0, K - 1, K // 2, 0, 0]
    for i in range(8):
        u[i, :K] = -rng.random(K)
        target[i, at[i], tokens[i, at[i]]] = 0.0
    u[6, 0] = -np.inf
    u[7, 0] = -0.0
    for d in (draft, None):
        want = [P.verify(target[i], None if d is None else d[i], tokens[i], u[i]) for i in range(8)]
        assert [m for m, _ in want] == at
        assert _verify(target, d, tokens, u) == want


def test_acceptance_border_and_zero_probabilities():
    p = np.zeros((5, 2, 40), np.float32)
    q = np.zeros((5, 1, 40), np.float32)
    p[:, 0, :2], p[:, 1, 5] = 0.5, 1.0
    p[:, 0, 1] = 0.25
    q[:, 0, 0] = [1.0, 1.0, 0.0, 0.0, 0.5]
    u = np.array([[0.5, 0.5], [np.nextafter(np.float32(0.5), np.float32(0)), 0.5], [0.9, 0.5], [0.9, 0.5], [0.99, 0.5]], np.float32)
    tokens = np.array([[0], [0], [0], [7], [0]], np.int32)
    # u q = p: rejected; just below: kept; q = 0 < p: kept; p = q = 0: rejected; p = q: kept for u < 1
    assert _verify(p, q, tokens, u) == [(0, 1), (1, 5), (1, 5), (0, 0), (1, 5)]


def test_nothing_left_takes_the_largest_probability():
    V = 5000
    p = np.full((3, 2, V), 1e-6, np.float32)
    q = np.full((3, 1, V), 1e-3, np.float32)
    p[0, 0, [17, 4000]] = 5e-4          # a tie: the lowest
    p[1, 0, V - 1] = 5e-4
    p[2] = 0.0
    assert _verify(p, q, [[3], [3], [3]], np.full((3, 2), 0.9, np.float32)) == [(0, 17), (0, V - 1), (0, 0)]


def test_counts_of_drafts_and_bad_tokens():
    rng = np.random.default_rng(4)
    target, draft, tokens, u = _random(rng, 8, 5, 600)
    u[:, :5] *= 0.5
    n = [0, 1, 2, 3, 4, 5, 5, 3]
    want = [P.verify(target[i, :n[i] + 1], draft[i, :n[i]], tokens[i, :n[i]], list(u[i, :n[i]]) + [u[i, 5]]) for i in range(8)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert _verify(target, draft, tokens, u, n_drafts=n, status=status) == want and int(status) == 0
    m = list(n)
    m[5], m[0] = 9, -3                   # clamped and reported
    assert _verify(target, draft, tokens, u, n_drafts=m, status=status) == want and int(status) == BAD_INDEX
    status.zero_()
    for bad in (-1, 600, 2 ** 31 - 1):
        t = tokens.copy()
        t[2, 0] = t[5, 2] = bad
        for d in (draft, None):
            status.zero_()
            want = [P.verify(target[i], None if d is None else d[i], t[i], u[i]) for i in range(8)]
            assert _verify(target, d, t, u, status=status) == want and int(status) == BAD_INDEX
            assert _verify(target, d, t, u) == want


def test_captured_and_on_two_streams():
    rng = np.random.default_rng(6)
    sets = [_random(rng, 5, 3, 40000) for _ in range(3)]
    want = [[P.verify(t[i], d[i], k[i], u[i]) for i in range(5)] for t, d, k, u in sets]
    dev = [[H.to_dev(x) for x in s] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[torch.zeros(5, dtype=torch.int32, device="cuda") for _ in range(2)] for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, d, o in zip(streams, dev, outs):
            Q.verify_drafts(*d, *o, stream=s)
    torch.cuda.synchronize()
    assert [list(zip(o[0].tolist(), o[1].tolist())) for o in outs] == want
    buf, out, g = [x.clone() for x in dev[0]], [torch.zeros_like(x) for x in outs[0]], torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        Q.verify_drafts(*buf, *out)
    for d, w in zip(dev, want):
        for b, x in zip(buf, d):
            b.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert list(zip(out[0].tolist(), out[1].tolist())) == w


def test_binding_refusals():
    t = torch.full((2, 3, 10), 0.1, device="cuda")
    k, u = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")
    a, b = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2))
    for args in ((t.half(), None, k, u, a, b), (t, t, k, u, a, b), (t, None, k.long(), u, a, b), (t, None, k, u[:, :2], a, b),
                 (t, None, k, u, a[:1], b), (t.cpu(), None, k, u, a, b), (t[:1].expand(2, 3, 10), None, k, u, a, b),
                 (t.transpose(1, 2), None, k, u, a, b)):
        with pytest.raises(ValueError):
            Q.verify_drafts(*args)
    with pytest.raises(Q.QsaError):
        many = torch.zeros(1, 66, 4, device="cuda")
        Q.verify_drafts(many, None, torch.zeros(1, 65, dtype=torch.int32, device="cuda"), torch.zeros(1, 66, device="cuda"), a[:1], b[:1])
    Q.verify_drafts(t[:0], None, k[:0], u[:0], a[:0], b[:0])


# ------------------------------------------------------------------ a layer's verification step

def test_rollback_of_rejected_drafts_on_the_device():
    """The multi-query step of a layer, verified and rolled back without the host: the state
    and the following steps equal the oracle's on the accepted tokens."""
    wl = synth.workload("tiny")
    T, vocab, n0 = 4, 211, 1018
    qsa = Q.Qsa(H.config_of(wl, max_ctx=1200))
    g = H.GpuLayer(qsa)
    ref = O.OracleLayer(O.QsaShape.of(wl), max_ctx=1200)
    pre = synth.prefill_tokens(wl, 0, n0)
    g.append(pre["k"], pre["v"], pre["idx"])
    g.update()
    ref.append_tokens(pre["k"], pre["v"], pre["idx"])
    ref.update_pooled_cache()
    rng = np.random.default_rng(0)
    acc, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    seen = set()
    for it in range(8):
        st = [synth.step_inputs(wl, 0, it * T + u) for u in range(T)]
        x = {k: np.stack([s[k] for s in st]) for k in st[0]}
        o = Q.alloc_multi_outputs(g.cfg, T)
        g.append(x["k"], x["v"], x["idx"])
        g.update()
        qsa.index_topk_multi(0, H.to_dev(x["q_idx"]), H.to_dev(x["w"].astype(np.float32)), o["sel"], o["n_sel"], o["scores"])
        qsa.sparse_attend_selected_multi(0, H.to_dev(x["q"]), o["sel"], o["n_sel"], o["out"])
        target, draft, tokens, u = _random(rng, 1, T - 1, vocab)
        u[:, :T - 1] *= rng.choice([0.0, 0.7, 1.0])
        Q.verify_drafts(*(H.to_dev(y) for y in (target, draft, tokens, u)), acc, nxt)
        qsa.rollback_rejected(0, T - 1, acc)
        m, t = P.verify(target[0], draft[0], tokens[0], u[0])
        ref.append_tokens(x["k"], x["v"], x["idx"])
        ref.update_pooled_cache()
        ref.rollback(ref.n - (T - 1) + m)
        assert (int(acc), int(nxt)) == (m, t)
        assert g.state() == (ref.n, ref.n // 4, 0)
        seen.add(m)
    assert len(seen) > 1
    g.update()
    ref.update_pooled_cache()
    H.assert_pooled_close(g.pooled_rows(0, ref.n // 4), ref.pooled.rows[:ref.n // 4])


def test_rollback_count_outside_the_drafts():
    wl = synth.workload("tiny")
    qsa = Q.Qsa(H.config_of(wl, max_ctx=64))
    g = H.GpuLayer(qsa)
    pre = synth.prefill_tokens(wl, 0, 22)
    for count, keep, code in ((0, 19, 0), (1, 20, 0), (3, 22, 0), (-2, 19, BAD_INDEX), (4, 22, BAD_INDEX)):
        qsa.restore_layer(0, 0, 0)
        g.append(pre["k"], pre["v"], pre["idx"])
        g.update()
        qsa.rollback_rejected(0, 3, torch.tensor([count], dtype=torch.int32, device="cuda"))
        assert g.state(clear=True) == (keep, min(keep // 4, 5), code)
    qsa.restore_layer(0, 2, 0)          # more drafts than tokens
    qsa.rollback_rejected(0, 5, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert g.state() == (0, 0, 0)
    with pytest.raises(Q.QsaError):
        qsa.rollback_rejected(0, -1, torch.zeros(1, dtype=torch.int32, device="cuda"))
