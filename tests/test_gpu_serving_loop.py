"""Serving with a bounded cache: scored stack steps, requests cut to their
heaviest tokens when they outgrow their budget, steps on what is left at the
rows' true positions, and tokens drawn with each row's own settings."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
import serving_reference as sref
from memory_bound_transformer_decode_gb300 import ddl
from test_gpu_kv8 import dev
from test_gpu_kv8_stack import Serving, config

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


class Bounded(Serving):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        cfg, S = self.cfg, self.per * self.page
        self.scores = [torch.full((self.R, cfg.H_kv, S), math.nan, device="cuda") for _ in range(cfg.layers)]
        n = ddl.ddl_stack_kv8_scored_workspace_bytes(self.shape, self.R, self.T, self.max_rows, S)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        self.gone = torch.zeros(self.R, dtype=torch.int32, device="cuda")  # tokens cut off so far

    def plan(self, add):
        ddl.ddl_page_plan(self.old, add, self.free[self.taken:], self.table, self.page, used=self.used,
                          status=self.status, **self.p)
        off = self.p["row_off"].long()
        gone = torch.repeat_interleave(self.gone, off[1:] - off[:-1])
        self.p["row_pos"][:gone.numel()] += gone  # rows go on at their true positions

    def step(self, add, x, decay=1.0, **opts):
        self.plan(add)
        ddl.ddl_stack_step_kv8_scored(self.shape, self.wtype, self.layers, self.pools, self.scores, decay,
                                      page_table=self.table, max_rows=self.max_rows, max_len=self.per * self.page,
                                      x_bf16=x, resid_out=self.res, out_bf16=self.out, bad=self.bad, workspace=self.ws,
                                      **self.p, **opts)

    def check_scores(self, before, decay):
        """The last layer's, whose q the workspace still holds."""
        cfg = self.cfg
        off, lens = self.p["row_off"].cpu().numpy(), self.p["kv_len"].cpu().numpy()
        at = ddl.ddl_workspace_view(self.shape, self.T, 1).q
        q = ddl.ws_tensor(self.ws, at, self.T * cfg.Nq).view(self.T, cfg.H_q, cfg.head_dim)
        table = self.table.cpu().numpy()
        _, lse, _, off_by = ref.attention(self.pools[-1], q, off, lens, table, cfg.head_dim ** -0.5)
        old = before.nan_to_num(nan=0.0)
        want, tol = sref.score(self.pools[-1], q, lse.nan_to_num(nan=0.0), off, lens, table, old, decay, cfg.head_dim ** -0.5)
        tol = tol + want * math.expm1(float(off_by.max()))  # (the step's lse is the attention's, not the exact one)
        got = self.scores[-1]
        for r, n in enumerate(lens):
            assert n == 0 or float(((got[r, :, :n].double() - want[r, :, :n]).abs() - tol[r, :, :n]).max()) <= 0

    def cut(self, keep, sinks, recent):
        """Every request over `keep` tokens cut to as many, in all layers."""
        lens = self.old.cpu().numpy()
        over = lens > keep
        new = torch.full_like(self.table, -1)
        z = torch.zeros(self.R, dtype=torch.int32, device="cuda")
        n = int(over.sum()) * keep
        i32 = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
        ddl.ddl_page_plan(z, dev(np.where(over, keep, 0)), self.free[self.taken:], new, self.page, row_off=i32(self.R + 1),
                          kv_len=i32(self.R), row_pos=i32(n), slot=i32(n), used=self.used, status=self.status)
        assert not self.status.any()
        self.taken += int(self.used)
        for l, pool in enumerate(self.pools):
            out = torch.full_like(self.scores[l], math.nan)
            kept = torch.full((self.R, self.cfg.H_kv, keep), -1, dtype=torch.int32, device="cuda")
            raw = [t.view(torch.uint8).cpu().numpy() if t.element_size() == 1 else t.double().cpu().numpy() for t in pool]
            want = sref.evict(raw[:2], raw[2:], self.scores[l].cpu().numpy(), lens, [keep] * self.R, self.table.cpu().numpy(),
                              new.cpu().numpy(), sinks, recent, self.page, self.codes == "int8", kept.cpu().numpy(),
                              out.cpu().numpy())
            ddl.ddl_kv8_evict(pool, self.scores[l], self.old, dev([keep] * self.R), self.table, new, self.per * self.page,
                              kept=kept, score_out=out, sinks=sinks, recent=recent, bad=self.bad)
            assert np.array_equal(kept.cpu().numpy(), want[2])
            assert np.array_equal(out.cpu().numpy(), want[3], equal_nan=True)
            live = new.cpu().numpy()[over].ravel()
            live = live[live >= 0]
            for i in range(2):
                got = pool[i].view(torch.uint8).cpu().numpy()[live]
                a, b = ref.decode(got, self.codes == "int8"), ref.decode(want[0][i][live], self.codes == "int8")
                assert np.array_equal(a, b, equal_nan=True)
            self.scores[l] = out
        o = dev(over.astype(int)).bool()
        self.gone += torch.where(o, self.old - keep, 0)
        self.table.copy_(torch.where(o[:, None], new, self.table))
        self.old.copy_(torch.where(o, keep, self.old))


@pytest.mark.parametrize("wtype,hd,T,codes", [(ddl.INT4, 64, 3, "int8"), (ddl.BF16, 128, 4, "e4m3"), (ddl.INT4, 128, 24, "e4m3")])
def test_a_bounded_cache(wtype, hd, T, codes):
    R, decay = 3, 0.75
    sv = Bounded(config(hd), wtype, R, T, 16, 24, codes, max_rows=T)
    g = np.random.RandomState(T)
    for i in range(14):
        add = g.multinomial(T, [1 / R] * R) if i < 8 else np.ones(R, int)
        x = torch.randn((T, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
        before = [tuple(t.clone() for t in p) for p in sv.pools]
        held = sv.scores[-1].clone()
        sv.step(dev(add), x, decay)
        torch.cuda.synchronize()
        sv.check(before, x)
        sv.check_scores(held, decay)
        sv.advance()
        if i in (4, 7, 10):
            sv.cut(keep=5 if T < 9 else 21, sinks=1, recent=2)
    assert int(sv.gone.min()) > 0
    # the step's hidden rows to tokens
    V = 1500
    head = ddl.ddl_pack_head((torch.randn((V, sv.cfg.D), device="cuda") * 0.2).bfloat16(), sv.cfg.D, V, ddl.BF16)
    logits = torch.zeros((R, V), device="cuda")
    best = ddl.ddl_lm_head(sv.cfg.D, V, ddl.BF16, head, sv.res[:R].contiguous(), logits=logits)
    t, k, p = [0.0, 0.8, 1.2], [0, 40, 0], [1.0, 0.95, 0.9]
    u = torch.tensor([0.3, 0.7, 0.95], device="cuda")
    f = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    tok = ddl.ddl_sample(logits, u, temperature=f(t), top_k=dev(k), top_p=f(p))
    assert int(tok[0]) == int(best[0])
    for b in range(R):
        assert int(tok[b]) in sref.draw(logits[b].double().cpu().numpy(), t[b], k[b], float(f(p)[b]), 0.0, float(u[b]))


def test_scored_steps_have_the_bits_of_plain_ones():
    plain, scored = (c(config(128), ddl.INT4, 3, 6, 16, 8, "e4m3", max_rows=6) for c in (Serving, Bounded))
    for a, b in zip(scored.pools, plain.pools):
        for s, t in zip(a, b):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
    for i, add in enumerate(([3, 2, 1], [1, 1, 4], [2, 2, 2], [1, 1, 1])):
        x = torch.randn((6, plain.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
        for sv in (plain, scored):
            sv.step(dev(add), x)
            sv.advance()
        n = sum(add)
        assert torch.equal(plain.res[:n], scored.res[:n]) and torch.equal(plain.out[:n], scored.out[:n])
    for l in range(2):  # every row of every step has given each query head a weight of 1
        total = scored.scores[l].nan_to_num(nan=0.0)
        rows = dev([7, 6, 8]).float()[:, None].expand(3, 2)
        assert torch.allclose(total.sum(-1), 4 * rows, rtol=1e-4)


def test_a_captured_loop():
    """Plan, scored step and draw in one graph, replayed while lengths move on."""
    sv = Bounded(config(64), ddl.INT4, 2, 2, 16, 4, "int8", max_rows=1)
    ev = Bounded(config(64), ddl.INT4, 2, 2, 16, 4, "int8", max_rows=1)
    for a, b in zip(sv.pools, ev.pools):
        for s, t in zip(a, b):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
    add, x = dev([1, 1]), torch.randn((2, sv.cfg.D), device="cuda").bfloat16()
    u, tok = torch.rand(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    k = dev([20, 0])

    def step(s, t):
        ddl.ddl_page_plan(s.old, add, s.free, s.table, s.page, used=s.used, status=s.status, **s.p)
        ddl.ddl_stack_step_kv8_scored(s.shape, s.wtype, s.layers, s.pools, s.scores, 0.5, page_table=s.table, max_rows=1,
                                      max_len=64, x_bf16=x, resid_out=s.res, workspace=s.ws, **s.p)
        ddl.ddl_sample(s.res, u, top_k=k, tokens=t)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [tuple(t.clone() for t in p) for p in sv.pools]
    with torch.cuda.stream(side):
        step(sv, tok)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(sv.pools, keep):
        for s, t in zip(a, b):
            s.copy_(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(sv, tok)
    want = torch.zeros_like(tok)
    for s in (sv, ev):
        for sc in s.scores:
            sc.zero_()
    for i in range(12):  # (one page holds them: the plan takes the same two pages whenever old is 0)
        x.copy_(torch.randn((2, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
        u.copy_(torch.rand(2, device="cuda"))
        graph.replay()
        step(ev, want)
        torch.cuda.synchronize()
        assert torch.equal(sv.res, ev.res) and torch.equal(tok, want)
        assert all(torch.equal(a, b) for a, b in zip(sv.scores, ev.scores))
        for s in (sv, ev):
            s.old.copy_(s.p["kv_len"])


def test_refusals():
    sv = Bounded(config(64), ddl.INT4, 2, 2, 16, 4, "e4m3", max_rows=1)
    x = torch.zeros((2, sv.cfg.D), dtype=torch.bfloat16, device="cuda")
    base = dict(page_table=sv.table, max_rows=1, max_len=64, x_bf16=x, out_bf16=sv.out, workspace=sv.ws, **sv.p)
    n = ddl.ddl_stack_kv8_workspace_bytes(sv.shape, 2, 2, 1, 64)
    for scores, decay, kw in ((sv.scores[:1], 1.0, {}), ([s[:, :, :63].contiguous() for s in sv.scores], 1.0, {}),
                              (sv.scores, 1.5, {}), (sv.scores, -0.5, {}), ([sv.scores[0], sv.scores[1][:1]], 1.0, {}),
                              ([s.half() for s in sv.scores], 1.0, {}), (sv.scores, 1.0, dict(workspace=sv.ws[:n]))):
        with pytest.raises((ValueError, ddl.DDLError)):
            ddl.ddl_stack_step_kv8_scored(sv.shape, sv.wtype, sv.layers, sv.pools, scores, decay, **{**base, **kw})
    torch.cuda.synchronize()


def test_a_captured_loop_that_cuts():
    """Plan, scored step, cut of the requests that outgrow their budget and draw in one graph without a number from
    the device: replayed, requests are cut time and again, and later rows attend to the new pages at their true
    positions, with the bits of the same calls made one by one."""
    R, T, page, per, budget, keep = 3, 4, 16, 4, 37, 21

    class Loop(Bounded):
        def __init__(self):
            super().__init__(config(64), ddl.INT4, R, T, page, per, "e4m3", max_rows=2)
            i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
            pages = 64  # more than the loop takes
            self.all_free, self.given = dev(np.random.RandomState(2).permutation(pages)), i32(1)
            self.window = self.all_free.clone()
            self.pools = [tuple(torch.zeros((pages, *t.shape[1:]), dtype=torch.uint8 if t.element_size() == 1 else t.dtype,
                                            device="cuda").view(t.dtype) for t in p) for p in self.pools]
            self.new, self.zero = i32(R, per), i32(R)
            self.cut_plan = dict(row_off=i32(R + 1), kv_len=i32(R), row_pos=i32(R * keep), slot=i32(R * keep))
            self.kept, self.cut_len = i32(R, self.cfg.H_kv, keep), i32(R)
            self.next_scores = [torch.zeros_like(s) for s in self.scores]
            for s in self.scores:
                s.zero_()
            self.at, self.tok = torch.arange(T, device="cuda", dtype=torch.int32), i32(T)

        def take(self):  # the free pages from the next one on
            self.given += self.used
            at = torch.arange(len(self.all_free), device="cuda") + self.given
            self.window.copy_(self.all_free[at.clamp(max=len(self.all_free) - 1)])

        def one(self, add, x, u):
            ddl.ddl_page_plan(self.old, add, self.window, self.table, page, used=self.used, status=self.status, **self.p)
            self.take()
            of = torch.searchsorted(self.p["row_off"][1:], self.at, right=True).clamp(max=R - 1)  # each row's request
            pos = self.p["row_pos"]
            pos.copy_(torch.where(pos >= 0, pos + self.gone[of], pos))
            ddl.ddl_stack_step_kv8_scored(self.shape, self.wtype, self.layers, self.pools, self.scores, 0.9,
                                          page_table=self.table, max_rows=2, max_len=per * page, x_bf16=x,
                                          resid_out=self.res, bad=self.bad, workspace=self.ws, **self.p)
            ddl.ddl_sample(self.res, u, tokens=self.tok)
            lens = self.p["kv_len"]
            over = lens > budget
            self.cut_len.copy_(torch.where(over, keep, -1))
            self.new.fill_(-1)
            ddl.ddl_page_plan(self.zero, torch.where(over, keep, 0).int(), self.window, self.new, page, used=self.used,
                              status=self.status, **self.cut_plan)
            self.take()
            for l, pool in enumerate(self.pools):
                self.next_scores[l].copy_(self.scores[l])
                ddl.ddl_kv8_evict(pool, self.scores[l], lens, self.cut_len, self.table, self.new, per * page, kept=self.kept,
                                  score_out=self.next_scores[l], sinks=2, recent=5, bad=self.bad)
                self.scores[l].copy_(self.next_scores[l])
            self.gone += torch.where(over, lens - keep, 0)
            self.table.copy_(torch.where(over[:, None], self.new, self.table))
            self.old.copy_(torch.where(over, keep, lens))

        def state(self):
            return [self.old, self.gone, self.table, self.given, self.window, *self.scores, *(t for p in self.pools for t in p)]

    sv, ev = Loop(), Loop()
    add, x, u = dev([1, 1, 1]), torch.zeros((T, sv.cfg.D), dtype=torch.bfloat16, device="cuda"), torch.zeros(T, device="cuda")
    start = [t.clone() for t in sv.state()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.one(add, x, u)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.one(add, x, u)
    for a, b in zip(sv.state(), start):
        a.copy_(b)
    total, g = np.zeros(R, int), np.random.RandomState(7)
    for i in range(60):
        n = np.array([1, 1, 2]) if i < 30 else g.permutation([0, 1, 2]) if i % 4 else np.array([1, 1, 1])
        add.copy_(dev(n))
        x.copy_(torch.randn((T, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
        u.copy_(torch.rand(T, generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
        graph.replay()
        ev.one(add, x, u)
        torch.cuda.synchronize()
        rows = int(n.sum())
        assert torch.equal(sv.res[:rows], ev.res[:rows]) and torch.equal(sv.tok[:rows], ev.tok[:rows]), i
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(sv.state(), ev.state())), i
        true = [p for r in range(R) for p in range(total[r], total[r] + n[r])]
        total += n
        assert sv.p["row_pos"][:rows].tolist() == true and (sv.p["row_pos"][rows:] == -1).all()
        assert np.array_equal(sv.old.cpu().numpy() + sv.gone.cpu().numpy(), total)
    assert int(sv.bad) == 0 and int(sv.gone.min()) > 0 and int(sv.given) <= 64 and (sv.gone > 32).any()
