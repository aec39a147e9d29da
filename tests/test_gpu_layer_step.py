"""The serving steps of a layer together, as a server calls them: block norms, quantised projections with the requests' adapters, rotation,
cache writes, windowed attention over blocks that come back to the pool. Every step's result is held against its 64-bit
definition over what the step before gave."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import layer_reference as L
from tests import paged_reference as R

pytestmark = pytest.mark.gpu

F32, F16, BF16, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int8
HQ, HKV, D, WIDTH, RANK, BLOCK, WINDOW, SINKS = 8, 4, 64, 512, 8, 16, 24, 3


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


class Layer:
    def __init__(self, C, requests, blocks, adapters, seed=0):
        self.C = C
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*s):
            return torch.randn(*s, generator=g, device="cuda")

        self.cb = O.analytic_codebook(4)
        self.outs = (HQ * D, HKV * D, HKV * D)
        self.w = [C.cq_encode(rand(o, WIDTH) * WIDTH ** -0.5, 4, self.cb) for o in self.outs]
        self.wo = C.cq_encode(rand(WIDTH, HQ * D) * (HQ * D) ** -0.5, 4, self.cb)
        n = max(adapters) + 1
        self.a = [(rand(n, RANK, WIDTH) * WIDTH ** -0.5).to(BF16) for _ in self.outs]
        self.b = [rand(n, o, RANK).to(BF16) for o in self.outs]
        self.ao, self.bo = [(rand(n, RANK, HQ * D) * (HQ * D) ** -0.5).to(BF16)], [rand(n, WIDTH, RANK).to(BF16)]
        self.scales = 0.2 * rand(n)
        self.who = adapters
        self.norm_w, self.post_w, self.qn, self.kn = 1 + 0.1 * rand(WIDTH), 1 + 0.1 * rand(WIDTH), rand(D), rand(D)
        self.rates = C.cq_rope_init(D)
        self.geom = C.cq_kv_geometry(HQ, HKV, D, D, 4, 4, self.cb, self.cb, D ** -0.5)
        self.cap = blocks * BLOCK
        size = C.cq_packed_bytes(self.cap, HKV * D, 128, 4)
        self.k, self.v = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.lens, self.held = np.zeros(requests, dtype=np.int64), np.zeros(requests, dtype=np.int64)
        self.table = _i32(np.full((requests, 64), -1))
        self.free = list(range(blocks))[::-1]

    def step(self, x, residual, new):
        """x fp32 [tokens, WIDTH]: what the layer before gave; the requests' new[s] tokens. Returns (residual, the layer's result)."""
        C, n = self.C, x.shape[0]
        room = len(self.free)
        plan = C.cq_kv_plan(_i32(self.lens), _i32(new), _i32(self.held), self.table, _i32(self.free + [0]), _i32([room]), BLOCK, n)
        cu, cu_host = plan["cu_new"], np.concatenate([[0], np.cumsum(new)])
        self.held = plan["held_out"].cpu().numpy().astype(np.int64)
        assert int(plan["n_free_out"]) >= 0
        self.free = self.free[:int(plan["n_free_out"])]
        # the residual stream, and the quantised activations of its norm
        res, xq, s = C.cq_block_norm(x, residual, self.norm_w, post_norm=True, branch_weight=self.post_w, branch_scale=0.5, out_dtype=I8)
        r, y, er, ey = L.block_norm(_np(x), _np(residual), _np(self.norm_w), post=True, wb=_np(self.post_w), branch=0.5, eps=np.float64(np.float32(1e-6)))
        assert (np.abs(_np(res) - r) <= L.rounded(r, er, "bfloat16")).all()
        codes, scale = _np(xq), _np(s)[:, None]
        assert (np.abs(codes * scale - y) <= scale * (0.5 + 2.0 ** -16) + ey).all()
        # projections and their adapters
        qkv = C.cq_gemm_grouped([{"blob": w, "out": o, "in": WIDTH, "bits": 4, "codebook": self.cb, "Xq": xq, "x_scale": s}
                                 for w, o in zip(self.w, self.outs)])
        before = [_np(t) for t in qkv]
        C.cq_lora_add(qkv, xq, self.a, self.b, _i32(self.who), cu, scales=self.scales, x_scale=s)
        for got, (o, e) in zip(qkv, L.lora(before, codes, [_np(a) for a in self.a], [_np(b) for b in self.b], self.who, cu_host, _np(self.scales),
                                           None, _np(s))):
            assert (np.abs(_np(got) - o) <= e).all()
        q, k = C.cq_qk_norm_rope(qkv[0].view(n, HQ, D), qkv[1].view(n, HKV, D), plan["positions"], self.rates, self.qn, self.kn, q_dtype=F16)
        C.cq_kv_write_slots(self.geom, self.k, self.v, self.cap, k, qkv[2], plan["slots"])
        o = C.cq_kv_window_attend(self.geom, q, self.k, self.v, self.cap, self.table, BLOCK, _i32(self.lens), cu, None, int(max(new)), WINDOW, SINKS)
        table, rows, sees = self.table.cpu().numpy().astype(np.int64), [], []
        for i, (l, m) in enumerate(zip(self.lens, new)):
            t = np.arange(l + m)
            t = t[(t < SINKS) | (t > l - WINDOW)]
            rows.append(table[i, t // BLOCK] * BLOCK + t % BLOCK)
            at = l + np.arange(m)[:, None]
            sees.append((t[None] <= at) & ((t[None] < SINKS) | (at - t[None] < WINDOW)))
        want, bound = L.attend_rows(_np(q), self.k.cpu().numpy(), self.v.cpu().numpy(), self.cap, rows, sees, cu_host, (HQ, HKV, D, D), 4, 4, self.cb, self.cb,
                                    np.float64(np.float32(D ** -0.5)))
        assert (np.abs(_np(o) - want) <= bound + 2.0 ** -11 * (np.abs(want) + bound) + 2.0 ** -25).all()
        # the output projection and its adapters
        oq, so = C.cq_act_quant_int8(o.float().view(n, -1))
        z = C.cq_gemm(self.wo, WIDTH, HQ * D, 4, self.cb, oq, so)
        zb = _np(z)
        C.cq_lora_add([z], oq, self.ao, self.bo, _i32(self.who), cu, scales=self.scales, x_scale=so)
        (zr, ze), = L.lora([zb], _np(oq), [_np(self.ao[0])], [_np(self.bo[0])], self.who, cu_host, _np(self.scales), None, _np(so))
        assert (np.abs(_np(z) - zr) <= ze).all()
        self.lens = self.lens + np.asarray(new)
        self.give_back()
        C.cq_device_status()
        return res, z

    def give_back(self):
        """Blocks that no later token can see go back to the pool."""
        table = self.table.cpu().numpy()
        for s, l in enumerate(self.lens):
            for b in range(int(self.held[s])):
                if table[s, b] >= 0 and b * BLOCK >= SINKS and (b + 1) * BLOCK <= l - WINDOW + 1:
                    self.free.append(int(table[s, b]))
                    table[s, b] = -1
        self.table = _i32(table)


def test_layer_step(C):
    """Prompts of uneven length, one of them in two chunks, then single tokens, from a pool that holds far fewer rows than the requests have
    tokens: what lies behind the windows is used again."""
    adapters = [1, -1, 0]
    layer = Layer(C, 3, 22, adapters)
    g = torch.Generator(device="cuda").manual_seed(7)
    steps = [[60, 5, 33], [50, 0, 0], [1, 1, 1], [1, 1, 0], [40, 1, 12]] + [[1, 1, 1]] * 20 + [[30, 70, 20], [1, 0, 1]]
    assert np.sum(steps, axis=0).max() > 150 and sum(np.sum(steps, axis=0)) > 22 * BLOCK
    for new in steps:
        n = sum(new)
        x = torch.randn(n, WIDTH, generator=g, device="cuda")
        residual = torch.randn(n, WIDTH, generator=g, device="cuda").to(BF16)
        res, z = layer.step(x, residual, new)
        final = C.cq_block_norm(z, res, layer.norm_w, post_norm=True, branch_weight=layer.post_w, gate=torch.randn(n, 1, generator=g, device="cuda"),
                                gate_act="sigmoid", out_dtype=F32)[1]
        assert torch.isfinite(final).all()


def test_layer_step_of_one_request_does_not_see_the_others(C):
    """The same request alone and in a batch: the same residuals, codes and (but for the order of sums) results."""
    x, residual = torch.randn(40, WIDTH, device="cuda"), torch.randn(40, WIDTH, device="cuda").to(BF16)
    batch, alone = Layer(C, 2, 16, [0, 1]), Layer(C, 1, 16, [0])
    alone.a, alone.b, alone.ao, alone.bo, alone.scales = batch.a, batch.b, batch.ao, batch.bo, batch.scales
    alone.w, alone.wo, alone.norm_w, alone.post_w, alone.qn, alone.kn = batch.w, batch.wo, batch.norm_w, batch.post_w, batch.qn, batch.kn
    r2, z2 = batch.step(x, residual, [25, 15])
    r1, z1 = alone.step(x[:25].contiguous(), residual[:25].contiguous(), [25])
    assert torch.equal(r1, r2[:25])
    assert ((z1 - z2[:25]).norm() / z1.norm()) < 0.02
