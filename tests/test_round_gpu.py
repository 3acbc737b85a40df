"""One speculative round through the operators as a server would chain them (needs an MI355X): a prompt's keys and
values appended to the paged cache, the outcome cache's guesses and the drafted chain as one tree, their rows scored
over the shared context, the chain verified from the resulting probabilities, and the next round on the longer context."""
import numpy as np
import pytest
import torch

from lossless_speculative_sampling_amd import capi

pytestmark = pytest.mark.gpu

V, E, HQ, HKV, D, PAGE, K = 512, 96, 8, 2, 64, 16, 4


class Model:
    """One attention layer between an embedding and a head: enough for tokens to depend on their whole context."""

    def __init__(self):
        g = torch.Generator().manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.emb, self.head = r(V, E), r(HQ * D, V) / 8
        self.w = [r(E, h * D) / E ** 0.5 for h in (HQ, HKV, HKV)]
        self.freqs = torch.tensor(capi.spec_rope_frequencies(D, 10000.0, 4.0), dtype=torch.float64)

    def qkv(self, tokens):
        x = self.emb[tokens.cpu()]
        return [(x @ w).to(torch.bfloat16).view(-1, w.shape[1] // D, D).cuda() for w in self.w]

    def dense(self, tokens):
        """The last token's attention over a plain sequence, in float64 from the same bf16 projections."""
        q, k, v = (x.cpu().double() for x in self.qkv(torch.tensor(tokens)))
        ang = torch.arange(len(tokens)).double()[:, None] * self.freqs
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        turn = lambda x: torch.cat([x[..., :D // 2] * c - x[..., D // 2:] * s, x[..., D // 2:] * c + x[..., :D // 2] * s], -1)  # noqa: E731
        q, k = turn(q).to(torch.bfloat16).double()[-1], turn(k).to(torch.bfloat16).double()
        k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
        w = torch.softmax((k * q).sum(-1) * D ** -0.5, 0)
        return (w[..., None] * v).sum(0), (w[..., None] * v.abs()).sum(0)


def test_a_round_from_the_prompt_to_the_next():
    m = Model()
    rng = np.random.default_rng(0)
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    ctx_tokens = [rng.integers(0, V, n).tolist() for n in (37, 5, 64)]
    B, pages = len(ctx_tokens), 40
    cache = capi.KVCache(*(torch.full((pages, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    rotary = capi.Rotary(m.freqs.cuda())
    order = rng.permutation(pages)
    table = order[:B * 8].reshape(B, 8)                      # room for 128 tokens of each request
    spare = (order[B * 8:, None] * PAGE + np.arange(PAGE)).reshape(-1)
    slot_of = lambda b, t: table[b][t // PAGE] * PAGE + t % PAGE  # noqa: E731
    # prompts
    for b, toks in enumerate(ctx_tokens):
        q, k, v = m.qkv(torch.tensor(toks))
        t = np.arange(len(toks))
        capi.spec_kv_append(k, v, i32(t), i32(slot_of(b, t)), cache, rotary)
    for round_ in range(2):
        ctx = np.array([len(x) for x in ctx_tokens])
        # the drafted chain and the guessed outcomes behind each of its depths, from the draft's own logits
        draft_logits = torch.randn((B, K + 1, V), generator=torch.Generator().manual_seed(round_)).cuda() * 2
        drafted = torch.softmax(draft_logits[:, :K], -1).reshape(B * K, V).multinomial(1).view(B, K).to(torch.int32)
        guesses, fan = capi.saguaro_cache_build(draft_logits, K, drafted, 9, 0.7, 1.0)
        hang = np.repeat(np.arange(K + 1), fan) - 1          # a guess for depth k follows drafted token k - 1
        tokens = torch.cat([drafted, guesses], 1).contiguous()
        parents = np.concatenate([np.arange(K) - 1, hang])
        N = tokens.shape[1]
        # a drafted token takes the slot it would have in the context; guesses take spare slots
        slots = np.stack([np.concatenate([[slot_of(b, ctx[b] + j) for j in range(K)], spare[b * 9:b * 9 + 9]]) for b in range(B)])
        rows = capi.spec_tree_rows(tokens, i32(np.tile(parents, (B, 1))), i32(slots), i32(ctx), K + 1)
        q, k, v = m.qkv(tokens.reshape(-1).clamp(min=0).long())
        q = capi.spec_kv_append(k, v, rows.positions.view(-1), rows.append_slots.view(-1), cache, rotary, q=q)
        out, _ = capi.spec_prefix_attention(q, cache, i32(table), i32(ctx), i32(np.arange(B + 1) * N),
                                            suffix_slots=rows.suffix_slots.view(B * N, K + 1), suffix_len=rows.suffix_len.view(-1))
        # every node against plain attention over its own path
        for b in range(B):
            for n in range(N):
                path, x = [], n
                while x >= 0:
                    path.append(int(tokens[b, x]))
                    x = parents[x]
                want, size = m.dense(ctx_tokens[b] + path[::-1])
                # weights and result rounded to bf16, rotated queries and keys to bf16 on both sides (a value next
                # to the middle of two may go either way: 2^-8 of a score of at most ~8, on a few of them)
                assert ((out[b * N + n].cpu().double() - want).abs() <= 2.0 ** -8 * (want.abs() + 3 * size) * 1.05).all(), (b, n)
        # the last context token's row gives q_0: verified from probabilities with the server's own random numbers
        last = [m.qkv(torch.tensor(x))[0][-1:] for x in ctx_tokens]
        lastq = capi.spec_kv_append(None, None, i32(ctx - 1), None, None, rotary, q=torch.cat(last))
        first, _ = capi.spec_prefix_attention(lastq, cache, i32(table), i32(ctx), i32(np.arange(B + 1)))
        scored = torch.cat([first[:, None], out.view(B, N, HQ, D)[:, :K]], 1).float().reshape(B, K + 1, HQ * D)
        target = torch.softmax(scored @ m.head.cuda(), -1)
        r = capi.spec_verify_probs(torch.softmax(draft_logits[:, :K], -1), target, drafted, torch.rand((B, K), device="cuda"),
                                   torch.rand(B, device="cuda"))
        assert (r.status == 0).all()
        slot, hit, _ = capi.saguaro_cache_lookup(0, guesses.contiguous(), fan, K, B, r.k, r.tstar)
        for b in range(B):
            n = int(r.k[b]) + 1
            new = r.emitted[b, :n].tolist()
            assert all(t >= 0 for t in new) and (r.emitted[b, n:] == -1).all() and new[:-1] == drafted[b, :n - 1].tolist()
            # accepted tokens lie where the context wants them; t* is put there
            t = ctx[b] + n - 1
            _, k1, v1 = m.qkv(torch.tensor([new[-1]]))
            capi.spec_kv_append(k1, v1, i32([t]), i32([slot_of(b, t)]), cache, rotary)
            ctx_tokens[b] += new
