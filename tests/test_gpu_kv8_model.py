"""The backbone over the paged 8-bit cache: what it writes against the bf16 path's K and V, its outputs against a plain
forward pass of the model in 64 bits with the same rounding points, and rows forked, moved and captured in between."""
import math

import pytest
import torch

import kv8_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def hra():
    import qwen3_prefill_delayed_gb300 as h
    h.lib()
    return h


@pytest.fixture(scope="module")
def model(hra):
    import workloads as W
    d = W.tiny_dims()
    w = W.make_backbone(d, 11)
    wg = {"embed": w["embed"].cuda(), "final_norm": w["final_norm"].cuda(),
          "layers": [{k: v.cuda() for k, v in l.items()} for l in w["layers"]]}
    return d, w, hra.Backbone(d, wg)


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def rounded(x):
    return x.to(BF16).double()


def norm(x, g, eps):
    return rounded(x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * g.double())


def rope(x, pos, theta):
    hd = x.shape[-1]
    f = theta ** (-torch.arange(0, hd, 2, dtype=torch.float64) / hd)
    a = pos[:, None].double() * f
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def plain(d, w, x, cache, new, start):
    """Packed rows x (float64, bf16 values) through every layer; appends to the CPU cache.  -> final-norm rows."""
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    pos = torch.cat([torch.arange(s, s + n) for s, n in zip(start, new)])
    T, nq, nkv, hd, eps = x.shape[0], d.n_q_heads, d.n_kv_heads, d.head_dim, d.rms_eps
    for l, lw in enumerate(w["layers"]):
        m = {k: v.double() for k, v in lw.items()}
        qkv = rounded(norm(x, m["attn_norm"], eps) @ m["w_qkv"].T).view(T, nq + 2 * nkv, hd)
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
        unit = lambda y, g: y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * g  # noqa: E731
        q = rounded(rope(unit(q, m["q_norm"]), pos, d.rope_theta))
        k = rounded(rope(unit(k, m["k_norm"]), pos, d.rope_theta))
        R.append(cache, l, k, v, cu, start)
        a, _ = R.attend(cache, l, q, cu, [s + n for s, n in zip(start, new)])
        x = rounded(x + rounded(a).reshape(T, nq * hd) @ m["w_o"].T)
        gu = norm(x, m["mlp_norm"], eps) @ m["w_gate_up"].T
        gate, up = rounded(gu[:, :d.ffn]), rounded(gu[:, d.ffn:])
        x = rounded(x + rounded(gate / (1 + (-gate).exp()) * up) @ m["w_down"].T)
    return norm(x, w["final_norm"], eps)


def close(got, want):
    """One bf16 step of K or V (a different order of fp32 sums) moves an E4M3 code by a whole step, 2^-3 of it, about one
    time in 2^4: the bar of the path's other E4M3 variant past its first quantisation."""
    a, b = got.double().cpu(), want.double()
    cos = float((a * b).sum() / (a.norm() * b.norm()))
    err = float((a - b).abs().max())
    assert err <= 0.3 and 1 - cos <= 1e-3, f"max|err| {err:.3g}, 1 - cos {1 - cos:.3g}"


def paged(hra, d, rows, n_slots, n_pages, lens_room, page_size=16):
    kv = hra.Kv8Cache.new(d, rows, n_slots, n_pages=n_pages, page_size=page_size)
    kv.update(room=i32(lens_room).cuda())
    return kv


def cpu(kv):
    return {"codes": kv.codes.cpu(), "scales": kv.scales.cpu(), "table": kv.page_table.cpu(), "lens": kv.lens.cpu(),
            "refs": kv.refs.cpu()}


LENS = [13, 1, 40, 97]


@pytest.mark.parametrize("full", [False, True])
def test_prefill(hra, model, full):
    d, w, bb = model
    g = torch.Generator().manual_seed(5)
    toks = torch.randint(0, d.vocab, (4, 100), generator=g, dtype=torch.int32)
    kv = paged(hra, d, 4, 128, 20, LENS)
    before = cpu(kv)
    out = bb.prefill(toks.cuda(), LENS, kv, full_last_layer=full)
    torch.cuda.synchronize()
    assert kv.device_error() == 0 and hra.hra_device_error(bb.last_ws) == 0
    assert kv.lens.cpu().tolist() == LENS
    # layer 0's K and V do not depend on the cache: those of the bf16 path, quantised
    bf = hra.new_kv_cache(d, 4, 128, fill=0.0)
    bb.prefill(toks.cuda(), LENS, bf)
    want = {k: v.clone() for k, v in before.items()}
    cu = [0]
    for n in LENS:
        cu.append(cu[-1] + n)
    k = torch.cat([bf[0, b, 0, :, :n].transpose(0, 1).cpu() for b, n in enumerate(LENS)])
    v = torch.cat([bf[0, b, 1, :, :n].transpose(0, 1).cpu() for b, n in enumerate(LENS)])
    R.append(want, 0, k, v, cu, [0] * 4)
    assert torch.equal(kv.codes[0].cpu(), want["codes"][0]) and torch.equal(kv.scales[0].cpu(), want["scales"][0])
    x = torch.cat([w["embed"][toks[b, :n].long()] for b, n in enumerate(LENS)]).double()
    hid = plain(d, w, x, before, LENS, [0] * 4)
    close(out, hid[[c - 1 for c in cu[1:]]])


def test_chunks_and_decode(hra, model):
    """A prompt in two chunks beside a running row, then single tokens with host and device positions."""
    d, w, bb = model
    g = torch.Generator().manual_seed(6)
    kv = paged(hra, d, 2, 128, 20, [100, 60])
    c = cpu(kv)
    start = [0, 0]
    for new in ([30, 17], [41, 1]):
        toks = torch.randint(0, d.vocab, (2, 50), generator=g, dtype=torch.int32)
        out = bb.prefill(toks.cuda(), new, kv, start_pos=start)
        x = torch.cat([w["embed"][toks[b, :n].long()] for b, n in enumerate(new)]).double()
        hid = plain(d, w, x, c, new, start)
        close(out, hid[[new[0] - 1, sum(new) - 1]])
        start = [s + n for s, n in zip(start, new)]
    pos = i32(start).cuda()
    for step in range(3):
        emb = torch.randn(2, d.hidden, generator=g).mul(0.05).to(BF16)
        want = plain(d, w, emb.double(), c, [1, 1], start)
        if step == 0:
            out = bb.decode(emb.cuda(), start, kv)
            pos += 1
        else:
            out = bb.decode_dev(emb.cuda(), pos, 127, kv)
        close(out, want)
        start = [s + 1 for s in start]
    assert pos.cpu().tolist() == start and kv.lens.cpu().tolist() == start
    assert kv.device_error() == 0


def test_forked_and_compacted_rows_go_on_alike(hra, model):
    """Rows that are copies of one another give the same bits on the same input, and moving pages changes none."""
    d, w, bb = model
    g = torch.Generator().manual_seed(7)
    toks = torch.randint(0, d.vocab, (2, 40), generator=g, dtype=torch.int32).cuda()
    kv = paged(hra, d, 4, 96, 40, [37, 21, 0, 0])
    bb.prefill(toks, [37, 21], kv)
    kv.update(i32([1, 0, 0, 1]).cuda(), i32([30] * 4).cuda())
    assert kv.lens.cpu().tolist() == [21, 37, 37, 21]
    assert int((kv.refs == 2).sum()) == 37 // 16 + 21 // 16
    pos = [21, 37, 37, 21]
    for step in range(12):
        e = torch.randn(2, d.hidden, generator=g).mul(0.05).to(BF16).cuda()
        out = bb.decode(e[[1, 0, 0, 1]], pos, kv)
        pos = [p + 1 for p in pos]
        assert torch.equal(out[0], out[3]) and torch.equal(out[1], out[2])
    emb = torch.randn(4, d.hidden, generator=g).mul(0.05).to(BF16).cuda()
    a = bb.decode(emb, pos, kv).clone()
    kv.update(i32([0, -1, 2, 3]).cuda())          # row 1 ends: its pages leave holes
    pages = kv.page_table.clone()
    kv.compact()
    assert not torch.equal(pages, kv.page_table)
    b = bb.decode(emb, [pos[0], 0, pos[2], pos[3]], kv)      # the same positions again
    torch.cuda.synchronize()
    for row in (0, 2, 3):
        assert torch.equal(a[row], b[row])
    assert kv.device_error() == hra.DEVERR_PAGE_RANGE        # row 1 owns no page


def test_audio_loop_in_a_graph(hra, model):
    """Frames replayed from one graph give the codes and the cache of eager frames."""
    import workloads as W
    d, _, bb = model
    audio = W.make_audio(d, torch.Generator().manual_seed(8))
    head = hra.AudioHead(d, audio["head_w"].cuda(), audio["code_emb"].cuda())
    toks = torch.randint(0, d.vocab, (3, 30), generator=torch.Generator().manual_seed(9), dtype=torch.int32).cuda()
    lens = [30, 7, 16]
    codes, caches = [], []
    for graph in (False, True):
        kv = paged(hra, d, 3, 96, 30, [n + 12 for n in lens])
        hid = bb.prefill(toks, lens, kv)
        loop = hra.ARLoop(bb, head, kv, hid, lens, pos_bound=95)
        if graph:
            loop.capture(12)
            loop.replay()
            codes.append(loop.codes_seq.clone())
        else:
            codes.append(torch.stack([loop.frame()[0].clone() for _ in range(12)]))
        torch.cuda.synchronize()
        assert kv.device_error() == 0 and kv.lens.cpu().tolist() == [n + 12 for n in lens]
        caches.append(kv)
    assert torch.equal(codes[0], codes[1])
    assert torch.equal(caches[0].codes, caches[1].codes) and torch.equal(caches[0].scales, caches[1].scales)


def test_refusals(hra, model):
    d, _, bb = model
    toks = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    kv = paged(hra, d, 2, 32, 4, [8, 8])
    emb = torch.zeros(2, d.hidden, dtype=BF16, device="cuda")
    with pytest.raises(hra.HraError):
        bb.prefill(toks, [8, 8], kv, start_pos=[0, 25])           # past the row's positions
    with pytest.raises(hra.HraError):
        bb.decode(emb, [0, 32], kv)
    with pytest.raises(hra.HraError):
        bb.decode_dev(emb, i32([0, 0]).cuda(), 32, kv)
    with pytest.raises(hra.HraError):
        bb.prefill(torch.zeros(3, 8, dtype=torch.int32, device="cuda"), [8, 8, 8], kv)
    with pytest.raises(hra.HraError):
        bb.prefill(toks, [8, 8], kv, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    import dataclasses
    for other in (dataclasses.replace(d, n_layers=1), dataclasses.replace(d, n_kv_heads=1), dataclasses.replace(d, head_dim=128)):
        with pytest.raises(hra.HraError):
            bb.decode(emb, [0, 0], hra.Kv8Cache.new(other, 2, 32))
