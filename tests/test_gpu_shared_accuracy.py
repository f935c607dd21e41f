"""Decode attention over a shared prefix where its roundings count: a first token that holds most of the weight and has
no value, and keys far from zero; each output element against softmax attention in 64 bits over the dequantised latents.

Bar: 2e-3 of the row's largest value, the decode attention's own, and half a step of bf16 (2^-8 of the value)."""
import numpy as np
import pytest

from gpu_helpers import dev, kept_wup, synthetic_latents, torch_mod
from test_gpu_shared_prefix import _codec, _queries, _sides

pytestmark = pytest.mark.gpu


def _with_latents(s, n_prefix, own, lat, seed):
    """Cache whose sequences share the latents `lat` [n_prefix P][n_eff] and hold own[b] [n][n_eff] of their own."""
    torch = torch_mod()
    import spectral_transform_coding_b200 as st
    codec, P, B = s["codec"], s["P"], len(own)
    extra = max([1] + [-(-len(x) // P) for x in own])
    ids = np.random.default_rng(seed).permutation(n_prefix + B * extra).astype(np.int32)
    table = np.concatenate([np.tile(ids[:n_prefix], (B, 1)), ids[n_prefix:].reshape(B, extra)], 1)
    cache = st.LatentCache(codec, batch=B, max_pages_per_seq=n_prefix + extra, n_pages=ids.size, device=dev(),
                           page_table=torch.from_numpy(table))
    codec.quantize_append(cache, torch.from_numpy(lat).to(dev()), torch.zeros(len(lat), dtype=torch.int32, device=dev()))
    cache.lengths.fill_(n_prefix * P)
    rows, seqs = np.concatenate(own), np.concatenate([np.full(len(x), b, np.int32) for b, x in enumerate(own)])
    if len(rows):
        codec.quantize_append(cache, torch.from_numpy(rows).to(dev()), torch.from_numpy(seqs).to(dev()))
    codec.device_status()
    return cache, table, torch.from_numpy(ids[:n_prefix]).to(dev()), cache.lengths.cpu().numpy()


def _two_bf16(W):
    """W as the fold of the queries takes it: two bf16 parts, 2^-17 of each entry left out."""
    torch = torch_mod()
    x = torch.from_numpy(np.ascontiguousarray(W, np.float32))
    hi = x.to(torch.bfloat16).float()
    return (hi.double() + (x - hi).to(torch.bfloat16).double()).numpy()


def _bar(s, cache, table, lengths, q, outs, fold=lambda W: W):
    """Largest error of each of `outs` [batch][heads][d_head] in units of the bar."""
    W = [[fold(K), V] for K, V in kept_wup(s["W_up"], s["widths"], s["group"])]
    gq = s["n_q"] // s["n_kv"]
    s.pop("pool", None)
    worst = np.zeros(len(outs))
    for b in range(len(lengths)):
        for a in range(s["n_kv"]):
            (cK, _), (cV, _) = _sides(s, cache, table, lengths, b, a)
            for h in range(a * gq, (a + 1) * gq):
                sc = cK @ (np.asarray(W[a][0], np.float64) @ q[b, h]) / np.sqrt(s["d_h"])
                w = np.exp(sc - sc.max())
                ref = (w / w.sum() @ cV) @ np.asarray(W[a][1], np.float64)
                bar = 2.0 ** -8 * np.abs(ref) + 2e-3 * np.abs(ref).max()
                for i, out in enumerate(outs):
                    off = np.abs(out[b, h] - ref) / bar
                    worst[i] = max(worst[i], float(off.max()) if np.isfinite(off).all() else np.inf)
    return worst


@pytest.mark.parametrize("batch", [1, 9])
@pytest.mark.parametrize("nats", [13.0, 15.5, 17.0])
def test_a_first_token_with_most_of_the_weight_and_no_value(nats, batch):
    """28,672 shared tokens with scores of deviation about 1; the first token's is `nats`, so that it takes between 0.8
    and 0.999 of the weight, and its value is zero: the output is what the other tokens' small weights leave."""
    torch = torch_mod()
    s = _codec("qwen8x", 21)
    P, n_prefix = s["P"], 448
    rng = np.random.default_rng(22)
    lat = rng.standard_normal((n_prefix * P, s["codec"].n_eff)).astype(np.float32)
    lat[:, 0] = 0.0
    lat[0] = 0.0
    W0 = np.asarray(kept_wup(s["W_up"], s["widths"], s["group"])[0][0][0], np.float64)  # K coordinate 0
    g = rng.standard_normal((batch, s["n_q"], s["d_h"])) * 1.4
    g += (8.0 - g @ W0)[..., None] * W0 / (W0 @ W0)
    lat[0, 0] = nats * np.sqrt(s["d_h"]) / 8.0
    q = torch.from_numpy(g.astype(np.float32)).to(dev()).to(torch.bfloat16)
    cache, table, prefix, lengths = _with_latents(s, n_prefix, [lat[:0]] * batch, lat, 23)
    out = s["codec"].decode_attend_shared(cache, q, prefix)
    s["codec"].device_status()
    (cK, _), (cV, _) = _sides(s, cache, table, lengths, 0, 0)
    assert np.all(cV[0] == 0) and np.count_nonzero(cK[0]) == 1
    rows = slice(0, 1) if batch == 1 else slice(0, 9, 8)
    worst = _bar(s, cache, table[rows], lengths[rows], q.double().cpu().numpy()[rows], [out.double().cpu().numpy()[rows]])
    assert worst[0] <= 1.0


@pytest.mark.parametrize("name", ["llama4x", "qwen8x", "g8wide", "allwidths"])
def test_keys_far_from_zero(name):
    """Keys with a common offset of many times their spread, as a projection with a bias gives them: the shared decode,
    the same with fewer pages shared, and the decode that shares nothing are all within the bar."""
    torch = torch_mod()
    s = _codec(name, 31)
    codec, P = s["codec"], s["P"]
    n_prefix = -(-400 // P)
    rng = np.random.default_rng(32)
    off = rng.choice([-50.0, 50.0], codec.n_eff).astype(np.float32)
    kept = kept_wup(s["W_up"], s["widths"], s["group"])
    col = 0
    for a in range(s["n_kv"]):  # (the value columns stay where they are)
        col += len(kept[a][0])
        off[col:col + len(kept[a][1])] = 0.0
        col += len(kept[a][1])
    assert col == codec.n_eff
    make = lambda n, k: synthetic_latents(n, codec.n_eff, seed=33 + k, decay=0.2) + off  # noqa: E731
    cache, table, prefix, lengths = _with_latents(s, n_prefix, [make(100, 1), make(0, 2)], make(n_prefix * P, 0), 34)
    q, q64 = _queries(s, 2, 35, scale=1.0)
    outs = [codec.decode_attend_shared(cache, q, prefix), codec.decode_attend_shared(cache, q, prefix[:n_prefix // 2]),
            codec.decode_attend(cache, q.float())]
    codec.device_status()
    worst = _bar(s, cache, table, lengths, q64, [o.double().cpu().numpy() for o in outs])
    assert worst[2] <= 1.0
    assert worst[1] <= 1.0
    assert worst[0] <= 1.0


@pytest.mark.parametrize("name", ["llama4x", "qwen8x", "allwidths"])
def test_keys_that_differ_by_most_of_the_range_of_fp16(name):
    """The last kept group of keys (1 bit; allwidths: also 8 bits) with spreads of about 60,000, and queries nearly
    orthogonal to it. Queries' low parts end at 2^-25: 2^-25 * 16 * 30000 / sqrt(128) = 1.3e-3 in a score at most. The
    fold's parts of W_up leave 2^-17 * 16 * 30000 * sum_d |q_d W_kd| (about 0.3) / sqrt(128) = 0.1 at most, several 1e-3
    in this case (the products of one sign cancel, what is left of them does not): the reference takes the same parts."""
    s = _codec(name, 51)
    codec, P = s["codec"], s["P"]
    kept = kept_wup(s["W_up"], s["widths"], s["group"])
    lat = synthetic_latents(6 * P, codec.n_eff, seed=52, decay=0.2)
    rng = np.random.default_rng(53)
    q, col = rng.standard_normal((2, s["n_q"], s["d_h"])), 0
    gq = s["n_q"] // s["n_kv"]
    for a in range(s["n_kv"]):
        nK, g = len(kept[a][0]), s["group"]
        lat[:, col + nK - g:col + nK] = rng.uniform(-30000, 30000, (len(lat), g))
        W = np.asarray(kept[a][0][nK - g:], np.float64)
        rows = slice(a * gq, (a + 1) * gq)
        q[:, rows] -= (q[:, rows] @ W.T) @ W
        col += nK + len(kept[a][1])
    torch = torch_mod()
    q = torch.from_numpy((0.05 * q).astype(np.float32)).to(dev()).to(torch.bfloat16)
    cache, table, prefix, lengths = _with_latents(s, 6, [lat[5:40], lat[:0]], lat, 54)
    out = codec.decode_attend_shared(cache, q, prefix)
    codec.device_status()
    assert _bar(s, cache, table, lengths, q.double().cpu().numpy(), [out.double().cpu().numpy()], _two_bf16)[0] <= 1.0


@pytest.mark.parametrize("own", [[0, 0], [0, 7], [70, 0]])
def test_a_nan_query_gives_nan_with_and_without_own_tokens(own):
    torch = torch_mod()
    s = _codec("qwen8x", 41)
    n_eff = s["codec"].n_eff
    lat = synthetic_latents(4 * s["P"], n_eff, seed=42)
    cache, _, prefix, _ = _with_latents(s, 4, [synthetic_latents(n, n_eff, seed=43 + n) for n in own], lat, 44)
    q, _ = _queries(s, 2, 45)
    want = s["codec"].decode_attend_shared(cache, q, prefix)
    q[0, 2] = float("nan")
    got = s["codec"].decode_attend_shared(cache, q, prefix)
    s["codec"].device_status()
    assert torch.isnan(got[0, 2]).all()
    keep = torch.ones_like(got[:, :, 0], dtype=torch.bool)
    keep[0, 2] = False
    assert torch.equal(got[keep], want[keep])
