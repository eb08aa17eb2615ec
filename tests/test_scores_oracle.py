"""Pins of the token-score and embedding-dropout oracle: against torch's
log_softmax and autograd in fp64, central differences, and the generator's
published known-answer vectors."""
import numpy as np
import pytest
import torch

from oracle import scores_oracle as S


def _case(seed, s=6, V=37):
    r = np.random.default_rng(seed)
    z = r.normal(0, 3, (s, V))
    z[1, 5:9] = -np.inf
    z[2, 3] = z[2, 11] = z[2, 20] = z[2].max() + 1.0          # ties at the top
    y = r.integers(0, V, s)
    y[1], y[3] = 0, -100
    return z, y


@pytest.mark.parametrize("T", [1.0, 0.6, 2.5])
def test_scores_match_log_softmax(T):
    z, y = _case(1)
    got = S.token_scores(z, y, top=5, temperature=T)
    lp = torch.log_softmax(torch.from_numpy(z) / T, dim=1).numpy()
    live = y != -100
    rows = np.nonzero(live)[0]
    np.testing.assert_allclose(got["logp"][live], lp[rows, y[live]], rtol=0, atol=1e-12)
    ent = torch.special.entr(torch.from_numpy(np.exp(lp))).sum(1).numpy()
    np.testing.assert_allclose(got["entropy"][live], ent[live], rtol=0, atol=1e-12)
    assert got["logp"][3] == got["entropy"][3] == 0 and np.all(got["top_ids"][3] == -1)
    assert list(got["top_ids"][2][:3]) == [3, 11, 20]
    for r in rows:
        np.testing.assert_allclose(got["top_logp"][r], np.sort(lp[r])[::-1][:5], rtol=0, atol=1e-12)
    np.testing.assert_allclose(got["stats"][live, 0] / T + got["stats"][live, 1],
                               torch.logsumexp(torch.from_numpy(z) / T, 1).numpy()[live], rtol=0, atol=1e-12)


def test_scores_gradient_matches_autograd_and_differences():
    z, y = _case(2)
    r = np.random.default_rng(3)
    s, V = z.shape
    T = 1.4
    gl, ge, gt = r.normal(size=s), r.normal(size=s), r.normal(size=(s, 4))
    ids = S.token_scores(z, y, top=4)["top_ids"]
    d = S.token_scores_backward(z, y, gl, ge, ids, gt, T)
    x = torch.from_numpy(z).requires_grad_()
    live = torch.from_numpy(y != -100)
    lp = torch.log_softmax(x / T, 1)
    p = lp.exp()
    ent = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1)
    pick = lp.gather(1, torch.from_numpy(np.maximum(y, 0))[:, None])[:, 0]
    alt = lp.gather(1, torch.from_numpy(np.maximum(ids, 0)))
    total = (torch.from_numpy(gl) * pick + torch.from_numpy(ge) * ent)[live].sum() \
        + (torch.from_numpy(gt) * alt)[live].sum()
    total.backward()
    ref = torch.nan_to_num(x.grad).numpy()
    np.testing.assert_allclose(d, ref, rtol=0, atol=1e-10)

    def value(zz):
        o = S.token_scores(zz, y, temperature=T)
        v = (gl * o["logp"] + ge * o["entropy"]).sum()
        for q in range(s):
            if y[q] != -100:
                u = zz[q] / T
                v += (gt[q] * (u - np.log(np.exp(u - u.max()).sum()) - u.max())[ids[q]]).sum()
        return v

    for q, k in [(0, 0), (0, int(y[0])), (2, 3), (4, 7), (1, 20)]:
        e = np.zeros_like(z)
        e[q, k] = 1e-5
        assert abs((value(z + e) - value(z - e)) / 2e-5 - d[q, k]) < 1e-7


def test_rows_without_a_distribution():
    z = np.array([[-np.inf] * 4, [0, np.inf, 1, np.inf], [1, np.nan, 2, -np.nan], [-np.inf, 1, -np.inf, -np.inf]])
    o = S.token_scores(z, np.array([0, 0, 0, 1]), top=4)
    assert np.isnan(o["logp"][:3]).all() and np.isnan(o["entropy"][:3]).all() and np.isnan(o["stats"][:3, 1]).all()
    assert o["top_ids"].tolist() == [[0, 1, 2, 3], [1, 3, 2, 0], [1, 3, 2, 0], [1, 0, 2, 3]]
    assert o["logp"][3] == 0 and o["entropy"][3] == 0 and np.isneginf(o["top_logp"][3, 1:]).all()
    d = S.token_scores_backward(z, np.array([0, 0, 0, 1]), g_entropy=np.ones(4))
    assert np.isnan(d[:3]).all() and np.all(d[3] == 0)


def test_philox_known_answers():
    def words(c, k):
        return [int(v) for v in S.philox4x32_10(c, k)]

    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert words((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_keeps_the_right_share_and_scales():
    keep = S.keep_mask(12345, 7, 400, 250, 0.3)
    n = keep.size
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / n)
    assert not np.array_equal(keep, S.keep_mask(12345, 8, 400, 250, 0.3))
    assert not np.array_equal(keep, S.keep_mask(12346, 7, 400, 250, 0.3))
    assert np.array_equal(keep[:100, :99], S.keep_mask(12345, 7, 100, 99, 0.3))   # of (row, column) alone
    table = np.random.default_rng(0).normal(size=(9, 10))
    out, bad = S.embedding_dropout_forward(table, [3, 8, -1, 9, 2], 2.0, 0.0, padding_id=2)
    assert bad and np.array_equal(out[:2], 2 * table[[3, 8]]) and not out[2:].any()


def test_embedding_gradient_is_the_adjoint():
    r = np.random.default_rng(5)
    V, h, s = 11, 13, 40
    ids = r.integers(-1, V + 1, s)
    kw = dict(scale=3.0, p=0.4, seed=99, offset=1 << 40, padding_id=4)
    E, g = r.normal(size=(V, h)), r.normal(size=(s, h))
    out, _ = S.embedding_dropout_forward(E, ids, **kw)
    d, mag, count = S.embedding_dropout_backward(g, ids, V, **kw)
    assert abs((out * g).sum() - (E * d).sum()) < 1e-10      # linear in E
    assert not d[4].any() and count[4] == 0 and np.all(mag >= np.abs(d) - 1e-12)
