"""The layer stack on 8-bit paged caches (ddl_page_plan -> ddl_stack_step_kv8):
prompts, decode and padding rows in one step, on each of the library's weight
paths, against the layer's formulas in 64 bits.

The appended codes are checked against the quantizer's definition on the
reference's own k and v; the attention of the reference reads the codes the
device holds, so that a code that falls the other way at a rounding border
(k and v are rounded to bf16 from values that differ by fp32 errors) does not
count twice.  Outputs meet the stack's bars: relative L2 2e-3 of the bf16
output, 2e-2 absolute of the fp32 residual.
"""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from gpu_helpers import MAX_ABS, REL_L2, rel_l2
from memory_bound_transformer_decode_gb300 import configs, ddl, synth, workload
from test_gpu_kv8 import CODES, dev, make_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ddl.load(build_if_missing=True)


def config(hd, layers=2, H_q=8, H_kv=2):
    return configs.DecodeConfig(f"kv8-hd{hd}", D=256, H_q=H_q, H_kv=H_kv, head_dim=hd, d_ff=320, rope_base=1e4,
                                kv_len=1, layers=layers, seed=31)


class Serving:
    def __init__(self, cfg, wtype, R, T, page, per, codes, max_rows):
        self.cfg, self.wtype, self.R, self.T, self.page, self.per, self.codes = cfg, wtype, R, T, page, per, codes
        self.max_rows, self.shape = max_rows, ddl.make_shape(cfg)
        self.layers, self.w64 = [], []
        for l in range(cfg.layers):
            w = synth.layer_weights(cfg, l, device="cuda")
            self.layers.append({"packed": workload.pack_layer_from_master(self.shape, wtype, w), "norm1": w["norm1"],
                                "norm2": w["norm2"]})
            self.w64.append({n: self._dense(w[n]) if n in workload.MATS else w[n].double() for n in w})
        self.pools = [make_pool(R * per, cfg.H_kv, page, cfg.head_dim, codes, seed=l, junk=True)
                      for l in range(cfg.layers)]
        self.free = dev(np.random.RandomState(5).permutation(R * per))
        self.table, self.old, self.taken = dev(np.full((R, per), -1)), dev(np.zeros(R)), 0
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.p = {"row_off": i32(R + 1), "kv_len": i32(R), "row_pos": i32(T), "slot": i32(T)}
        self.used, self.status, self.bad = i32(1), i32(R), i32(1)
        n = ddl.ddl_stack_kv8_workspace_bytes(self.shape, R, T, max_rows, per * page)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # (NaN everywhere)
        self.out = torch.empty((T, cfg.D), dtype=torch.bfloat16, device="cuda")
        self.res = torch.empty((T, cfg.D), dtype=torch.float32, device="cuda")

    def _dense(self, w):
        if self.wtype == ddl.BF16:
            return w.double()
        q, s = ddl.ddl_quantize_int4(w)
        lo, hi = (q & 15).short(), (q >> 4).short()
        c = torch.stack([lo, hi], -1).reshape(w.shape)
        c = torch.where(c > 7, c - 16, c).double()
        return (c.view(w.shape[0], -1, 64) * s.double()[..., None]).view(w.shape)

    def step(self, add, x, **opts):
        ddl.ddl_page_plan(self.old, add, self.free[self.taken:], self.table, self.page, used=self.used,
                          status=self.status, **self.p)
        ddl.ddl_stack_step_kv8(self.shape, self.wtype, self.layers, self.pools, page_table=self.table,
                               max_rows=self.max_rows, max_len=self.per * self.page, x_bf16=x, resid_out=self.res,
                               out_bf16=self.out, bad=self.bad, workspace=self.ws, **self.p, **opts)

    def advance(self):
        self.taken += int(self.used)
        self.old.copy_(self.p["kv_len"])

    def check(self, before, x, softcap=0.0, window=0, slopes=None):
        """before: the pools ahead of the step."""
        cfg, hd = self.cfg, self.cfg.head_dim
        off, lens = self.p["row_off"].cpu().numpy(), self.p["kv_len"].cpu().numpy()
        slot, pos = self.p["slot"].cpu().numpy(), self.p["row_pos"].cpu().numpy()
        table = self.table.cpu().numpy()
        assert (self.status == 0).all() and int(self.bad) == 0
        n = int(off[-1])
        z = x[:n].double()
        ang = torch.from_numpy(pos[:n].astype(np.float64)).cuda()[:, None, None] * cfg.rope_base ** (
            -2.0 * torch.arange(hd // 2, device="cuda").double() / hd)

        def rope(t):
            a, b = t[..., :hd // 2], t[..., hd // 2:]
            return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)

        rms = lambda t, w: t * w / (t.pow(2).mean(-1, keepdim=True) + cfg.eps).sqrt()  # noqa: E731
        for l, w in enumerate(self.w64):
            h = rms(z, w["norm1"])
            q = rope((h @ w["wq"].T).view(n, cfg.H_q, hd))
            k, v = rope((h @ w["wk"].T).view(n, cfg.H_kv, hd)), (h @ w["wv"].T).view(n, cfg.H_kv, hd)
            # INT4 weights at 5 to 15 rows: the stage's input has fp16's 11 bits, each product within 2^-11 of
            # itself, and RoPE adds two such sums (|cos| + |sin| <= sqrt 2)
            wide = self.wtype == ddl.INT4 and 5 <= self.T <= 15
            for i, t, m in ((0, k, "wk"), (1, v, "wv")):
                err = (h.abs() @ w[m].abs().T).view(n, cfg.H_kv, 2, hd // 2).amax(2, keepdim=True).expand(
                    -1, -1, 2, -1).reshape(n, cfg.H_kv, hd).cpu().numpy() * (2.0 ** -11 * 2 ** 0.5 if wide else 0)
                codes, scale = ref.append(before[l][i].view(torch.uint8).cpu().numpy(),
                                          before[l][i + 2].cpu().numpy(), t.bfloat16().double().cpu().numpy(),
                                          slot[:n], self.page, self.codes == "int8")
                got = self.pools[l][i].view(torch.uint8).cpu().numpy()
                gs, off_t = self.pools[l][i + 2].cpu().numpy(), slot[:n] % self.page
                pg = slot[:n] // self.page
                a = ref.decode(got[pg, :, off_t], self.codes == "int8") * gs[pg, :, off_t // 16][..., None]
                b = ref.decode(codes[pg, :, off_t], self.codes == "int8") * scale[pg, :, off_t // 16][..., None]
                # k and v differ by the projection's fp32 error, 1e-4 of the rows' RMS (the bar of the bf16
                # rows), and a border then moves a value to the next code: one step of the larger scale
                top = np.maximum(gs, scale)[pg, :, off_t // 16][..., None]
                step = top if self.codes == "int8" else np.maximum(np.abs(a), np.abs(b)) / 8 + top / 512
                far = np.abs(a - b) > 1.001 * step + 2.0 ** -7 * np.abs(b) + 1e-4 * np.sqrt(np.mean(b * b)) + 1.2 * err
                assert not far.any(), (l, i, np.argwhere(far)[:8], a[far][:8], b[far][:8])
                assert ((a == b).mean()) > (0.9 if wide else 0.95)
            o, _, _, _ = ref.attention(self.pools[l], q, off, lens, table, hd ** -0.5, softcap, window, slopes)
            y = z + o.reshape(n, -1) @ w["wo"].T
            h2 = rms(y, w["norm2"])
            g = h2 @ w["wg"].T
            z = y + (g * torch.sigmoid(g) * (h2 @ w["wu"].T)) @ w["wd"].T
        assert rel_l2(self.out[:n].double().cpu(), z.cpu()) <= REL_L2
        assert float((self.res[:n].double() - z).abs().max()) <= MAX_ABS
        assert ddl.ddl_read_device_status(self.ws, self.shape, self.T, 1) == 0


CASES = [(ddl.INT4, 64, 1, "e4m3"), (ddl.INT4, 128, 3, "e4m3"), (ddl.INT4, 128, 2, "int8"), (ddl.BF16, 64, 4, "int8"),
         (ddl.BF16, 128, 1, "e4m3"), (ddl.INT4, 128, 9, "e4m3"), (ddl.INT4, 64, 15, "int8"),
         (ddl.INT4, 128, 24, "e4m3"), (ddl.BF16, 128, 12, "e4m3"), (ddl.BF16, 64, 64, "int8")]


@pytest.mark.parametrize("wtype,hd,T,codes", CASES)
def test_serving_steps(wtype, hd, T, codes):
    """Prompt rows, then decode rows, some of the T rows padding."""
    R = min(T, 4)
    sv = Serving(config(hd), wtype, R, T, 16, 12, codes, max_rows=T)
    g = np.random.RandomState(T)
    for i in range(5):
        add = np.ones(R, int) if i in (2, 4) else g.multinomial(T, [1 / R] * R) if i < 3 else g.randint(0, 2, R)
        x = torch.randn((T, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
        before = [tuple(t.clone() for t in p) for p in sv.pools]
        sv.step(dev(add), x)
        torch.cuda.synchronize()
        sv.check(before, x)
        sv.advance()


def test_attention_options_in_the_stack():
    sv = Serving(config(128, H_q=6), ddl.INT4, 3, 8, 32, 8, "e4m3", max_rows=8)
    slopes = torch.exp2(-torch.arange(6, device="cuda").float())
    for i, add in enumerate(([5, 2, 1], [1, 1, 1], [1, 6, 0], [1, 1, 1])):
        x = torch.randn((8, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
        before = [tuple(t.clone() for t in p) for p in sv.pools]
        sv.step(dev(add), x, softcap=20.0, window=9, slopes=slopes)
        torch.cuda.synchronize()
        sv.check(before, x, 20.0, 9, slopes)
        sv.advance()


@pytest.mark.parametrize("wtype,T", [(ddl.INT4, 2), (ddl.INT4, 6), (ddl.INT4, 20), (ddl.BF16, 8)])
def test_captured_step(wtype, T):
    """plan and stack step in one graph, replayed while lengths and pages move on; the same bits as eager steps."""
    sv, ev = (Serving(config(128), wtype, T, T, 16, 4, "e4m3", max_rows=1) for _ in range(2))
    for a, b in zip(sv.pools, ev.pools):
        for s, t in zip(a, b):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
    add = dev(np.ones(T))
    x = torch.randn((T, sv.cfg.D), device="cuda").bfloat16()
    free = sv.free.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [tuple(t.clone() for t in p) for p in sv.pools]
    with torch.cuda.stream(side):
        sv.step(add, x)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(sv.pools, keep):
        for s, t in zip(a, b):
            s.copy_(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.step(add, x)
    taken = 0
    for i in range(20):
        x.copy_(torch.randn((T, sv.cfg.D), generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
        graph.replay()
        ev.step(add, x)
        torch.cuda.synchronize()
        assert torch.equal(sv.res, ev.res) and torch.equal(sv.p["kv_len"], ev.p["kv_len"])
        taken += int(sv.used)
        sv.free.copy_(torch.roll(free, -taken))
        sv.old.copy_(sv.p["kv_len"])
        ev.advance()
    assert (sv.p["kv_len"] == 20).all() and int(sv.bad) == 0


def test_refusals():
    sv = Serving(config(64), ddl.INT4, 2, 2, 16, 4, "e4m3", max_rows=1)
    x = torch.zeros((2, sv.cfg.D), dtype=torch.bfloat16, device="cuda")
    base = dict(page_table=sv.table, max_rows=1, max_len=64, x_bf16=x, out_bf16=sv.out, workspace=sv.ws, **sv.p)

    def call(layers=None, pools=None, **kw):
        ddl.ddl_stack_step_kv8(sv.shape, sv.wtype, sv.layers if layers is None else layers,
                               sv.pools if pools is None else pools, **{**base, **kw})

    other = make_pool(8, 2, 32, 64, "e4m3")
    for kw in (dict(pools=sv.pools[:1]), dict(pools=[sv.pools[0], other]), dict(max_rows=65), dict(max_rows=0),
               dict(max_len=0), dict(workspace=sv.ws[:4096]), dict(x_bf16=x[:, :128].contiguous()),
               dict(x_bf16=x.float()), dict(slot=sv.p["slot"][:1]), dict(kv_len=sv.p["kv_len"].long()),
               dict(softcap=-1.0), dict(window=-2), dict(row_off=sv.p["row_off"][:2])):
        with pytest.raises((ValueError, ddl.DDLError)):
            call(**kw)
    torch.cuda.synchronize()
