"""The backbone over the paged 8-bit cache with a reach: every layer's attention through a window, and over prefixes that rows
share, against a plain forward pass of the model in 64 bits with the same rounding points."""
import pytest
import torch

import kv8_reach_ref as W
import kv8_ref as R
from test_gpu_kv8_model import BF16, close, cpu, hra, i32, model, paged, plain  # noqa: F401
from test_gpu_kv8_shared import wide

pytestmark = pytest.mark.gpu


def through(window, sinks, monkeypatch):
    """The plain pass (test_gpu_kv8_model.plain) with attention through a window."""
    monkeypatch.setattr(R, "attend", lambda c, l, q, cu, lens: W.attend(c, l, q, cu, lens, window, sinks))


@pytest.mark.parametrize("window,sinks", [(20, 3), (1, 0), (64, 16)])
def test_prompts_chunks_and_tokens_through_a_window(hra, model, monkeypatch, window, sinks):  # noqa: F811
    d, w, bb = model
    through(window, sinks, monkeypatch)
    g = torch.Generator().manual_seed(6)
    reach = hra.Kv8Reach(window=window, sinks=sinks)
    kv = paged(hra, d, 2, 160, 24, [0, 0])
    c = cpu(kv)
    start = [0, 0]
    for new in ([60, 17], [31, 1]):
        # the pages of the step: those that no later token sees go, and the plain pass keeps its own copy of what it wrote
        kv.update(room=i32(new).cuda(), reach=reach)
        c["table"] = merged(c["table"], kv.page_table.cpu())
        toks = torch.randint(0, d.vocab, (2, 60), generator=g, dtype=torch.int32)
        out = bb.prefill(toks.cuda(), new, kv, start_pos=start, reach=reach)
        x = torch.cat([w["embed"][toks[b, :n].long()] for b, n in enumerate(new)]).double()
        hid = plain(d, w, x, c, new, start)
        close(out, hid[[new[0] - 1, sum(new) - 1]])
        start = [s + n for s, n in zip(start, new)]
    pos = i32(start).cuda()
    for step in range(3):
        kv.update(room=i32([1, 1]).cuda(), reach=reach)
        c["table"] = merged(c["table"], kv.page_table.cpu())
        emb = torch.randn(2, d.hidden, generator=g).mul(0.05).to(BF16)
        want = plain(d, w, emb.double(), c, [1, 1], start)
        if step == 0:
            out = bb.decode(emb.cuda(), start, kv, reach=reach)
            pos += 1
        else:
            out = bb.decode_dev(emb.cuda(), pos, 159, kv, reach=reach)
        close(out, want)
        start = [s + 1 for s in start]
    assert kv.lens.cpu().tolist() == start and kv.device_error() == 0
    kv.update(reach=reach)                                      # what the last tokens have left behind goes too
    pages = sum(not W.gone(n, 16, window, sinks, i) for n in start for i in range(-(-n // 16)))
    assert int((kv.refs > 0).sum()) == pages


def merged(old, new):
    """The plain pass's table: new pages where there are any (it never looks at the others, which may have other owners)."""
    return torch.where(new >= 0, new, old)


def forked(hra, d, bb, rows, prompt, room, g):  # noqa: F811
    """`rows` continuations of one prompt, in a table so wide that its positions, as the bound of a prefix, are worth sharing."""
    P = 16
    width = wide(d.n_kv_heads, d.head_dim, P, rows, 1)
    kv = hra.Kv8Cache.new(d, rows, width * P, n_pages=64, page_size=P)
    kv.update(room=i32([prompt] + [0] * (rows - 1)).cuda())
    toks = torch.randint(0, d.vocab, (1, prompt), generator=g, dtype=torch.int32)
    bb.prefill(toks.cuda(), [prompt], kv)
    kv.update(i32([0] * rows).cuda(), i32([room] * rows).cuda())
    return kv


def test_continuations_of_one_prompt(hra, model):  # noqa: F811
    d, w, bb = model
    g = torch.Generator().manual_seed(6)
    rows, prompt = 4, 75
    kv = forked(hra, d, bb, rows, prompt, 40, g)
    reach = hra.Kv8Reach(groups=i32([0, rows]).cuda(), prefix=i32([prompt]).cuda(), max_own=40)
    c = cpu(kv)
    c["table"] = c["table"][:, :16].contiguous()
    start = [prompt] * rows
    for new in ([3, 1, 5, 2], [1, 6, 1, 4]):                    # a few tokens each
        toks = torch.randint(0, d.vocab, (rows, 6), generator=g, dtype=torch.int32)
        out = bb.prefill(toks.cuda(), new, kv, start_pos=start, reach=reach)
        x = torch.cat([w["embed"][toks[b, :n].long()] for b, n in enumerate(new)]).double()
        hid = plain(d, w, x, c, new, start)
        close(out, hid[[sum(new[:b + 1]) - 1 for b in range(rows)]])
        start = [s + n for s, n in zip(start, new)]
    pos = i32(start).cuda()
    counts = {}
    for step in range(4):
        emb = torch.randn(rows, d.hidden, generator=g).mul(0.05).to(BF16)
        want = plain(d, w, emb.double(), c, [1] * rows, start)
        before = hra.hra_launch_counter()
        if step < 2:
            out = bb.decode(emb.cuda(), start, kv, reach=reach if step else None)
            pos += 1
        else:
            out = bb.decode_dev(emb.cuda(), pos, 127, kv, reach=reach)
        counts[step] = hra.hra_launch_counter() - before
        close(out, want)
        start = [s + 1 for s in start]
    # one plan a pass, and in each layer the prefix, the rows' own positions and the join in the place of one kernel
    assert counts[1] - counts[0] == 1 + 2 * d.n_layers and counts[2] == counts[1]
    assert kv.lens.cpu().tolist() == start and kv.device_error() == 0


@pytest.mark.parametrize("kind", ["window", "groups"])
def test_audio_loop_in_a_graph(hra, model, kind):  # noqa: F811
    """Frames replayed from one graph give the codes and the cache of eager frames."""
    import workloads as Wl
    d, _, bb = model
    audio = Wl.make_audio(d, torch.Generator().manual_seed(8))
    head = hra.AudioHead(d, audio["head_w"].cuda(), audio["code_emb"].cuda())
    rows, prompt = 3, 37
    codes, caches = [], []
    for graph in (False, True):
        g = torch.Generator().manual_seed(5)
        kv = forked(hra, d, bb, rows, prompt, 14, g)
        if kind == "window":
            reach = hra.Kv8Reach(window=24, sinks=2)
        else:
            reach = hra.Kv8Reach(groups=i32([0, rows]).cuda(), prefix=i32([prompt]).cuda(), max_own=14)
        hid = torch.randn(rows, d.hidden, generator=g).to(BF16).cuda()
        loop = hra.ARLoop(bb, head, kv, hid, [prompt] * rows, pos_bound=63, reach=reach)
        if graph:
            loop.capture(12)
            loop.replay()
            codes.append(loop.codes_seq.clone())
        else:
            codes.append(torch.stack([loop.frame()[0].clone() for _ in range(12)]))
        torch.cuda.synchronize()
        assert kv.device_error() == 0 and kv.lens.cpu().tolist() == [prompt + 12] * rows
        caches.append(kv)
    assert torch.equal(codes[0], codes[1])
    assert torch.equal(caches[0].codes, caches[1].codes) and torch.equal(caches[0].scales, caches[1].scales)


def test_refusals(hra, model):  # noqa: F811
    d, _, bb = model
    kv = paged(hra, d, 2, 32, 4, [8, 8])
    emb = torch.zeros(2, d.hidden, dtype=BF16, device="cuda")
    toks = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    bf = hra.new_kv_cache(d, 2, 32, fill=0.0)
    w = hra.Kv8Reach(window=4)
    for call in (lambda: bb.prefill(toks, [8, 8], bf, reach=w), lambda: bb.decode(emb, [0, 0], bf, reach=w),
                 lambda: bb.decode_dev(emb, i32([0, 0]).cuda(), 8, bf, reach=w),
                 lambda: hra.ARLoop(bb, None, bf, emb, [0, 0], 8, reach=w)):
        with pytest.raises(hra.HraError, match="Kv8Cache"):
            call()
    many = hra.Kv8Reach(groups=i32([0, 1, 2, 2]).cuda(), prefix=i32([0, 0, 0]).cuda())      # more groups than rows
    with pytest.raises(hra.HraError):
        bb.prefill(toks, [8, 8], kv, reach=many)
    with pytest.raises(hra.HraError):
        bb.decode(emb, [0, 0], kv, reach=many)
    with pytest.raises(hra.HraError):
        kv.update(reach=hra.Kv8Reach(groups=i32([0, 2]).cuda(), prefix=i32([0]).cuda()))
    with pytest.raises(hra.HraError):
        kv.attend(0, toks, i32([0, 1]).cuda(), i32([1]).cuda(), 1, 1, reach=(4, 0))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(hra.HraError):
        bb.decode(emb, [0, 0], kv, workspace=ws, reach=w)


def test_group_arrays_inside_what_a_pass_writes_are_refused(hra, model):  # noqa: F811
    d, _, bb = model
    kv = paged(hra, d, 2, 32, 4, [8, 8])
    emb = torch.zeros(2, d.hidden, dtype=BF16, device="cuda")
    toks = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    bb.prefill(toks, [8, 8], kv)
    ws = torch.zeros(2 * bb.last_ws.numel() + (1 << 20), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, d.hidden, dtype=BF16, device="cuda")
    pos = i32([0, 0]).cuda()
    prefix = i32([0]).cuda()
    for groups in (ws[256:264].view(torch.int32), out.view(torch.int32).view(-1)[:2], pos):
        r = hra.Kv8Reach(groups=groups, prefix=prefix)
        with pytest.raises(hra.HraError):
            bb.decode_dev(emb, pos, 4, kv, out=out, workspace=ws, reach=r)
        if groups is not pos:
            with pytest.raises(hra.HraError):
                bb.decode(emb, [0, 0], kv, out=out, workspace=ws, reach=r)
            with pytest.raises(hra.HraError):
                bb.prefill(toks, [8, 8], kv, out=out, workspace=ws, reach=r)
    bb.decode_dev(emb, pos, 4, kv, out=out, workspace=ws, reach=hra.Kv8Reach(groups=i32([0, 2]).cuda(), prefix=prefix))


@pytest.mark.parametrize("rows,kernels", [(80, 1), (2, 0)])
def test_prompts_are_listed_once_a_pass(hra, model, rows, kernels):  # noqa: F811
    """Prompts of more (token, head) rows than a short sequence's tile has take the list's kernel, once, and no other more; a few
    of them do without it."""
    d, _, bb = model
    G = d.n_q_heads // d.n_kv_heads
    counts = []
    for n in (16 // G, 16 // G + 1):
        kv = paged(hra, d, rows, 32, 2 * rows, [16] * rows)
        toks = torch.zeros(rows, n, dtype=torch.int32, device="cuda")
        before = hra.hra_launch_counter()
        bb.prefill(toks, [n] * rows, kv, full_last_layer=True)
        counts.append(hra.hra_launch_counter() - before)
    assert d.n_layers > 1 and counts[1] - counts[0] == kernels
