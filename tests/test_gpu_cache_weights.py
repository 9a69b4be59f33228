"""The cache attention's weights and merges on the GPU, against bounds that do not grow with the
length (tests/cache_bounds.py): a key that takes nearly all of a row's weight, long sequences in which
every run of rows shows in the output."""
import numpy as np
import pytest
import torch

from tests import cache_bounds as cb
from tests.test_cache_bounds import SHARED

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _quantised(x):
    """(codes, scales [Hkv, blocks]) of x [L, Hkv, D], scales as the cache's."""
    L, H, D = x.shape
    nb = -(-L // 32)
    pad = np.concatenate([x, np.zeros((nb * 32 - L, H, D))]).reshape(nb, 32, H, D)
    amax = np.abs(pad).max((1, 3))                                       # [nb, H]
    s = np.exp2(np.ceil(np.log2(np.maximum(amax, 1e-30) / 448.0)).clip(-40, 40))
    codes = torch.from_numpy((pad / s[:, None, :, None]).reshape(-1, H, D)[:L]).float().to(torch.float8_e4m3fn)
    return codes, torch.from_numpy(s.T.copy()).float()


def _run(kind, seqs, B, **how):
    """A batch of B of the sequences (q, k, v) in turn. Returns the outputs of the first and the last of
    them (whose tiles are cut elsewhere), and for each what the kernel saw: q, k, v, value scales."""
    import target_model_verify_gb300 as tv
    L, Hkv, D = seqs[0][1].shape
    n, Hq = seqs[0][0].shape[:2]
    m = len(seqs)

    def many(t):
        return torch.cat([t.to(DEV)] * -(-B // m))[:B].contiguous()

    q = torch.stack([torch.from_numpy(s[0]).to(torch.bfloat16) for s in seqs])
    if kind == "masked":
        k, v = (torch.stack([torch.from_numpy(s[x]).to(torch.bfloat16) for s in seqs]) for x in (1, 2))
        seen = [(q[b].double().numpy(), k[b].double().numpy(), v[b].double().numpy(), None) for b in range(m)]
        cache = (many(k), many(v))
    else:
        ks, vs = [_quantised(s[1]) for s in seqs], [_quantised(s[2]) for s in seqs]
        at = np.arange(L) // 32
        seen = []
        for b in range(m):
            sk, sv = ks[b][1].double().numpy().T[at], vs[b][1].double().numpy().T[at]      # [L, Hkv]
            seen.append((q[b].double().numpy(), ks[b][0].double().numpy() * sk[..., None],
                         vs[b][0].double().numpy() * sv[..., None], sv))
        codes = [many(torch.stack([x[0].view(torch.uint8) for x in t])).view(torch.float8_e4m3fn) for t in (ks, vs)]
        cache = (*codes, *(many(torch.stack([x[1] for x in t])) for t in (ks, vs)))
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    if how.get("slopes") is not None:
        how = dict(how, slopes=torch.tensor(how["slopes"], dtype=torch.float32, device=DEV))
    ws = torch.empty(tv.cache_attention_workspace_bytes(B, n, Hq, Hkv, D, L), dtype=torch.uint8, device=DEV)
    fn = tv.verify_attention_masked if kind == "masked" else tv.verify_attention_kv8
    out = fn(many(q), *cache, lens, workspace=ws, **how)
    again = fn(many(q), *cache, lens, workspace=ws, **how)
    assert tv.read_status(ws) == 0
    assert torch.equal(out, again)
    rows = list(range(m)) + list(range(max(m, B - m), B))
    return out[rows].double().cpu().numpy(), [seen[b % m] for b in rows]


def _compare(kind, seqs, B, **how):
    got, seen = _run(kind, seqs, B, **how)
    for g, (q, k, v, sv) in zip(got, seen):
        want, tol = cb.outputs_and_bounds(kind, q, k, v, sv, **how)
        err = np.abs(g - want)
        assert (err <= tol).all(), (kind, float((err / tol).max()), float(err.max()), float(np.abs(want).max()))


@pytest.mark.parametrize("weight", [0.9, 0.98, 1 - 2.0 ** -10])
@pytest.mark.parametrize("kind,B,n,Hq,Hkv,D,L", [
    ("kv8", 32, 2, 16, 8, 128, 32768),         # many tiles: the cache on the M side
    ("kv8", 40, 2, 16, 8, 128, 4096),
    ("kv8", 3, 2, 16, 8, 128, 2000),           # few tiles: copies of the query rows
    ("kv8", 2, 10, 8, 2, 128, 9000),           # 40 query rows
    ("kv8", 2, 26, 8, 2, 64, 9000),            # 104 query rows, a lane each
    ("kv8", 2, 2, 8, 2, 256, 9000),
    ("masked", 8, 2, 16, 8, 128, 32768),
    ("masked", 2, 26, 8, 2, 64, 9000),
])
def test_one_key_with_nearly_all_the_weight(kind, B, n, Hq, Hkv, D, L, weight):
    """The first key takes `weight` of every row and has value 0: the output is what the other keys'
    small weights say."""
    rng = np.random.default_rng([B, D, L])
    _compare(kind, [cb.with_sink(rng, n, Hq, Hkv, D, L, weight) for _ in range(2)], B)


@pytest.mark.parametrize("weight", [0.999, 1 - 2.0 ** -14, 1 - 2.0 ** -20])
@pytest.mark.parametrize("kind,B,n,Hq,Hkv,D,L", [
    ("kv8", 40, 2, 16, 8, 128, 20000), ("kv8", 2, 2, 16, 8, 128, 9000), ("kv8", 2, 10, 8, 2, 128, 9000),
    ("kv8", 2, 26, 8, 2, 64, 20000), ("kv8", 2, 2, 8, 2, 256, 9000), ("masked", 2, 2, 16, 8, 128, 9000),
])
def test_equal_weights_beside_a_dominant_one(kind, B, n, Hq, Hkv, D, L, weight):
    """All other scores are equal, so that a rounding of their weights is the same for all and shows."""
    rng = np.random.default_rng([B, D, L, 1])
    _compare(kind, [cb.with_sink(rng, n, Hq, Hkv, D, L, weight, sigma=0.0) for _ in range(2)], B)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
def test_sharp_scores_and_a_sink(kind):
    """Scores of three times the spread: the references move both ways."""
    rng = np.random.default_rng(5)
    _compare(kind, [cb.with_sink(rng, 2, 16, 8, 128, 4096, 0.98, sigma=3.0) for _ in range(2)], 40)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,L", [(1, 2, 16, 8, 128, 40000), (40, 2, 16, 8, 128, 3000),
                                            (40, 2, 16, 8, 128, 500), (2, 4, 8, 2, 128, 3000)])
def test_sink_under_a_distance_bias(kind, B, n, Hq, Hkv, D, L):
    """Biases from flat to steep: references go down block by block, as far as they may."""
    rng = np.random.default_rng([B, L])
    slopes = np.exp2(-np.arange(Hq) * 0.75).astype(np.float32)
    _compare(kind, [cb.with_sink(rng, n, Hq, Hkv, D, L, 0.9) for _ in range(min(B, 2))], B, slopes=slopes)


@pytest.mark.parametrize("cap", [0.0, 1000.0])
@pytest.mark.parametrize("kind,B,D", [("kv8", 48, 64), ("kv8", 260, 128), ("masked", 48, 64)])
def test_exponents_of_millions(kind, B, D, cap):
    """Exponents of 2^24 and more, where fp32 has no fractions left: two equal scores, the second value
    under a scale of up to 2^8 times the first's. Outputs stay between the two values."""
    import target_model_verify_gb300 as tv
    L, lead = 160, 20
    q = torch.zeros(B, 1, 1, D)
    q[..., 0] = 128.0
    k = torch.zeros(B, L, 1, D)
    k[..., 0] = -448.0
    # odd sequences: all scores are negative
    big = torch.tensor([448.0, 416.0, 384.0, 352.0, 320.0, 288.0])[torch.arange(B) // 2 % 6]
    k[:, lead, 0, 0] = k[:, 128 + lead, 0, 0] = big * torch.tensor([1.0, -0.25])[torch.arange(B) % 2]
    up = torch.tensor([2.0 ** 8, 2.0 ** 7, 2.0 ** 6, 2.0 ** 3])[torch.arange(B) // 12 % 4]
    v = torch.zeros(B, L, 1, D)
    v[:, lead] = 1.0
    v[:, 128 + lead] = 2.0 if kind == "masked" else (2.0 / up)[:, None, None]
    sk, sv = torch.ones(B, 1, 5), torch.ones(B, 1, 5)
    sv[:, 0, 4] = up
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    q, k, v, sk, sv = (t.to(DEV) for t in (q, k, v, sk, sv))
    for scale in (2.0 ** 6, 2.0 ** 8, 2.0 ** 9, 2.0 ** 10, 2.0 ** 12):
        how = {"scale": scale, "softcap": cap}
        if kind == "masked":
            out = tv.verify_attention_masked(*(t.to(torch.bfloat16) for t in (q, k, v)), lens, **how)
        else:
            k8, v8 = (t.to(torch.float8_e4m3fn) for t in (k, v))
            out = tv.verify_attention_kv8(q.to(torch.bfloat16), k8, v8, sk, sv, lens, **how)
        assert out.isfinite().all(), (scale, out.isfinite().logical_not().nonzero()[:3])
        assert ((out >= (0 if cap else 1)) & (out <= 2)).all(), scale


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,L", [(1, *s) for s in SHARED] + [
    (3, 2, 8, 2, 128, 5000),        # three sequences over every CTA
    (40, 2, 16, 8, 128, 3000),      # more tiles than CTAs, cut anywhere
    (2, 4, 100, 100, 64, 1500),     # more heads than CTAs side by side
])
def test_every_part_of_a_shared_tile_reaches_the_output(kind, B, n, Hq, Hkv, D, L):
    """Values in which every 64 rows show (test_no_run_of_rows_can_be_lost_unnoticed)."""
    _compare(kind, [cb.with_marks(np.random.default_rng([n, L, b]), n, Hq, Hkv, D, L) for b in range(min(B, 2))], B)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("how", [{"window": 4000}, {"softcap": 20.0}, {"parent": (-1, 0, 0, 1), "window": 7001},
                                 {"scale": 0.03}], ids=str)
def test_shared_tiles_with_options(kind, how):
    _compare(kind, [cb.with_marks(np.random.default_rng(9), 4, 8, 2, 128, 9001)], 1, **how)
