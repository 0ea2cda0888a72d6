"""The decode-step calls as a serving program runs them: on streams, in captured graphs that nothing has warmed up, after a link, and
together with the batched calls as one captured decode loop."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from .test_gpu_batch import PAGE, i32, pkl, nothing_flagged, rope_table, rotated, sync  # noqa: F401  (fixtures)
from .test_gpu_batch_decode_loop import hold as hold_attention
from .test_gpu_step_rows import E4M3, check_norm, near, reference
from .test_gpu_weight4 import randn

pytestmark = pytest.mark.gpu


def hold_product(y, values, x, x_scales=None):
    """y against 64 bits of what the packed weights stand for: fp32 sums whose partial ones are larger than the result (see
    test_gpu_weight4): 2^-24 (sqrt(G) + 40) of the norm."""
    K = values.shape[1]
    X = x.double() if x_scales is None else x.double() * x_scales.double().repeat_interleave(128, dim=1)[:, :K]
    ref = X @ values.double().t()
    rel = ((y.double() - ref).norm() / ref.norm()).item()
    assert rel < 2.0 ** -24 * ((K / 64) ** 0.5 + 40), rel


@pytest.mark.parametrize("eight_bit", [False, True])
def test_captured_decode_loop(pkl, eight_bit):
    """Two layers of a decoder with 4-bit weights, from the token to the likeliest next one, captured once and replayed: lengths, tokens
    and hidden states stay on the device. Every call is held to its formula on what it was given."""
    H, G, D, d, ffn, V, n, layers, steps = 8, 2, 128, 1024, 2048, 4001, 3, 2, 20
    act = E4M3 if eight_bit else torch.float16
    W = lambda seed, N, K: pkl.pack_weight4((randn(seed, N, K) * K ** -0.5).bfloat16(), 64)  # noqa: E731
    qkv_w, o_w = [W(10 + l, (H + 2 * G) * D, d) for l in range(layers)], [W(20 + l, d, H * D) for l in range(layers)]
    gu_w, down_w, head = [W(30 + l, 2 * ffn, d) for l in range(layers)], [W(40 + l, d, ffn) for l in range(layers)], W(50, V, d)
    values = {id(w): pkl.unpack_weight4(w) for w in qkv_w + o_w + gu_w + down_w + [head]}
    gains, embed = [1 + 0.1 * randn(60 + i, d) for i in range(2 * layers + 1)], randn(70, V, d)
    rope, pool = rope_table(64, D), 16
    k = torch.zeros(layers, pool, G, PAGE, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table, kv, new = i32(np.full((n, 4), -1)), i32([0] * n), i32([1] * n)
    free = torch.arange(pool, dtype=torch.int32, device="cuda")
    bt = pkl.BlockTables(kv, i32([0] * n), i32([0] * (n + 1)), i32([0] * n), i32([-1] * n), i32([0, 0, 0]))
    token, seen = torch.tensor([3, 1000, 4000], dtype=torch.int32, device="cuda"), {}

    def norm(name, h, gain, delta):
        r = pkl.add_rms_norm(h, gain, delta, dtype=act)
        seen[name] = dict(h=h.clone(), y=r[0] if eight_bit else r, s=r[1] if eight_bit else None, gain=gain)
        return r if eight_bit else (r, None)

    def product(name, w, x, s=None):
        seen[name] = dict(w=w, x=x, s=s, y=pkl.gemm_w4(w, x, s))
        return seen[name]["y"]

    def step():
        pkl.block_tables(kv, new, table, free, n, free_used=bt.counts[1:2], out=bt)
        h, delta = embed[token.long()], None
        for l in range(layers):
            x, s = norm(f"attn{l}", h, gains[2 * l], delta)
            q = pkl.qk_norm_rope(product(f"qkv{l}", qkv_w[l], x, s), H, G, bt.row_pos, bt.row_slot, rope, k[l], v[l])
            a = pkl.attention_window(q, bt.row_start, pkl.BatchPages(kv, table), k[l], v[l], rope, 0)
            seen[f"att{l}"] = dict(q=q, a=a)
            delta = product(f"o{l}", o_w[l], a.view(n, H * D))
            x, s = norm(f"mlp{l}", h, gains[2 * l + 1], delta)
            gate, up = product(f"gu{l}", gu_w[l], x, s).chunk(2, dim=1)
            delta = product(f"down{l}", down_w[l], (gate * torch.sigmoid(gate) * up).half())
        x, s = norm("final", h, gains[-1], delta)
        seen["logits"] = product("head", head, x, s)
        seen["out"] = pkl.token_logprobs(seen["logits"], token, top=4)
        seen["token"] = token.clone()
        token.copy_(seen["out"].top_ids[:, 0])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        new.zero_()
        step()                                                # no rows: modules load, the token is put back below
    torch.cuda.synchronize()
    assert sync() == 0
    new.fill_(1), kv.zero_(), token.copy_(torch.tensor([3, 1000, 4000], dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    chosen = [[] for _ in range(n)]
    for t in range(steps):
        graph.replay()
        assert sync() == 0
        for l in range(layers):
            for name in (f"attn{l}", f"mlp{l}"):
                e = seen[name]
                check_norm(e["y"], e["s"], e["h"], e["gain"], 1e-5, act)
            for name in (f"qkv{l}", f"o{l}", f"gu{l}", f"down{l}"):
                e = seen[name]
                hold_product(e["y"], values[id(e["w"])], e["x"], e["s"])
            u = torch.arange(t + 1, device="cuda")
            for r in range(n):
                place = torch.tensor([int(table[r, i // PAGE]) * PAGE + i % PAGE for i in range(t + 1)]).cuda()
                K, Vv = (p[l][place // PAGE, :, place % PAGE].double() for p in (k, v))
                e = seen[f"att{l}"]
                hold_attention(e["a"][r:r + 1], e["q"][r:r + 1], rotated(K, u, rope), Vv, torch.ones(1, t + 1, dtype=torch.bool, device="cuda"), True)
        hold_product(seen["logits"], values[id(head)], seen["head"]["x"], seen["head"]["s"])
        lp, ent, ids, tops = reference(seen["logits"], seen["token"], 4)
        near(seen["out"].logprob, lp), near(seen["out"].entropy, ent), near(seen["out"].top_logprobs, tops)
        assert torch.equal(seen["out"].top_ids, ids) and torch.equal(token, ids[:, 0])
        for r in range(n):
            chosen[r].append(int(token[r]))
    assert kv.tolist() == [steps] * n and all(len(set(c)) > 1 for c in chosen)


def test_logprobs_of_a_link_and_a_decode(pkl):
    """LinkResult.logprobs and DecodeResult.logprobs: the query's own tokens scored, the next ones chosen."""
    import pic_inputs as pi
    wl = pi.config_workloads()["tiny"]
    model = pkl.PicModel(wl.spec, pi.gen_weights(wl.spec, gains="random"))
    store = pkl.PicStore(model, num_blocks=64, max_rows=512, max_requests=8, max_positions=1024)
    cids = store.compile(wl.chunks)
    req = wl.requests[0]
    res = store.link([([cids[c] for c in req.chunk_ids], req.query)], wl.k, all_logits=True)
    following = torch.tensor(np.append(req.query[1:], -1), dtype=torch.int32).cuda()          # the last row has none
    r = res.logprobs(following, top=3)
    store.sync()
    lp, ent, ids, tops = reference(res.logits, following.clamp(min=0), 3)
    near(r.logprob[:-1], (lp[0][:-1], lp[1][:-1]))
    assert torch.equal(r.top_ids[:-1], ids[:-1])
    last = res.logprobs(top=3)
    assert torch.equal(last.top_ids, ids) and last.logprob is None
    dec = store.decode(res.requests, [int(last.top_ids[-1, 0])])
    r = dec.logprobs(top=5)
    store.sync()
    lp, ent, ids, tops = reference(dec.logits, ids[:1, 0], 5)
    near(r.entropy, ent), near(r.top_logprobs, tops)
    assert torch.equal(r.top_ids, ids)
    store.close()
    model.close()


FIRST = """
import torch
import position_independent_kv_link_gb300 as pkl
torch.cuda.set_device(0)
T, e4m3 = %d, %r
N, K = 35000, 2048
codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda")
scales = torch.rand(N, K // 128, device="cuda").half()
h, delta, x = torch.randn(T, K, device="cuda"), torch.randn(T, K, device="cuda"), torch.randn(T, K, device="cuda")
tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
want = h + delta
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    w = pkl.pack_codes4(codes, scales)
    y = pkl.add_rms_norm(h, None, delta, dtype=torch.float8_e4m3fn if e4m3 else torch.float16)
    logits = pkl.gemm_w4(w, *y) if e4m3 else pkl.gemm_w4(w, y)
    r = pkl.token_logprobs(logits, tokens, 4)
    values = pkl.unpack_weight4(w)
    w2 = pkl.pack_weight4(values)
graph.replay()
pkl.sync()
assert torch.equal(h, want)
X = y[0].double() * y[1].double().repeat_interleave(128, 1) if e4m3 else y.double()
ref = X @ values.double().t()
assert ((logits.double() - ref).norm() / ref.norm()).item() < 3e-6
assert torch.equal(r.top_ids, torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :4].int())
assert torch.equal(values, scales.float().repeat_interleave(128, 1) * (codes.float() - 8))
print("captured")
"""


@pytest.mark.parametrize("T,e4m3", [(1, False), (5, True), (16, True), (40, False), (64, True)])
def test_first_calls_of_a_process_captured(pkl, T, e4m3):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (T, e4m3)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_streams(pkl):
    """On a stream that is not the current one: the call waits for what that stream was ordered behind, its results are of that
    stream's memory, and two streams at once do not meet."""
    N, K, T, V = 35000, 2048, 40, 50000
    codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda")
    w = pkl.pack_codes4(codes, torch.ones(N, K // 128, dtype=torch.float16, device="cuda"))
    xs = [randn(i, T, K).half() for i in range(4)]
    ls = [randn(10 + i, 9, V) for i in range(4)]
    hs = [randn(20 + i, 300, 4096) for i in range(4)]
    want = [(pkl.gemm_w4(w, x), pkl.token_logprobs(l, top=9), pkl.add_rms_norm(h.clone())) for x, l, h in zip(xs, ls, hs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        got = []
        for s, x, l, h in zip(streams, xs, ls, hs):
            got.append((pkl.gemm_w4(w, x, stream=s), pkl.token_logprobs(l, top=9, stream=s), pkl.add_rms_norm(h, stream=s)))
            junk = torch.full((T, N), 1e30, device="cuda")   # of the current stream: must not be given what the call still writes
            del junk
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1].top_ids, b[1].top_ids) and torch.equal(a[1].top_logprobs, b[1].top_logprobs)
            assert torch.equal(a[2], b[2])
    with pytest.raises(ValueError, match="stream"):
        pkl.gemm_w4(w, xs[0], out=torch.empty(T, N, device="cuda"), stream=type("S", (), {"device_index": 1, "cuda_stream": 0})())


def test_results_stay_with_the_stream(pkl):
    """Results that are dropped at once are not given to the current stream."""
    s = torch.cuda.Stream()
    codes = torch.randint(0, 16, (256, 256), dtype=torch.uint8, device="cuda")
    scales = torch.ones(256, 2, dtype=torch.float16, device="cuda")
    w = pkl.pack_codes4(codes, scales)
    h = randn(1, 8, 256)
    torch.cuda.synchronize()
    made = [pkl.pack_codes4(codes, scales, stream=s).data, pkl.pack_weight4(h, stream=s).data, pkl.unpack_weight4(w, stream=s),
            pkl.gemm_w4(w, h.half(), stream=s), *pkl.add_rms_norm(h, dtype=E4M3, stream=s), pkl.token_logprobs(h, top=3, stream=s).top_ids]
    sizes, addresses = [m.numel() * m.element_size() for m in made], [m.data_ptr() for m in made]
    del made
    taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    assert not {t.data_ptr() for t in taken} & set(addresses)
    s.synchronize()


def test_two_graphs(pkl):
    """Two captured steps replayed in turn, and at once on two streams."""
    N, K = 35000, 2048
    w = pkl.pack_codes4(torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda"), torch.ones(N, K // 128, dtype=torch.float16, device="cuda"))
    graphs = []
    for T in (1, 33):
        x = randn(T, T, K).half()
        y, g = torch.empty(T, N, device="cuda"), torch.cuda.CUDAGraph()
        pkl.gemm_w4(w, x, out=y)
        want = y.clone()
        r0 = pkl.token_logprobs(y, top=5)
        with torch.cuda.graph(g):
            pkl.gemm_w4(w, x, out=y)
            r = pkl.token_logprobs(y, top=5)
        graphs.append((g, y, want, r, r0))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for at_once in (False, True):
        for _ in range(4):
            for (g, y, want, r, r0), s in zip(graphs, streams):
                y.zero_()
            torch.cuda.synchronize()
            for (g, y, want, r, r0), s in zip(graphs, streams):
                if at_once:
                    with torch.cuda.stream(s):
                        g.replay()
                else:
                    g.replay()
            torch.cuda.synchronize()
            for g, y, want, r, r0 in graphs:
                assert torch.equal(y, want) and torch.equal(r.top_ids, r0.top_ids) and torch.equal(r.top_logprobs, r0.top_logprobs)
