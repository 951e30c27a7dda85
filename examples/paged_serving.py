"""A serving loop over the paged code cache: requests of different lengths come,
are prefilled in chunks, decode with drafted tokens that are partly rejected, and
leave; all of them share one pool of pages of 8-bit product-VQ codes.

    python examples/paged_serving.py [--steps 40] [--requests 12] [--scalar]

With --scalar the pages hold rotated keys and values as 4-bit scalar codes.  At the end half
of the seats go on as samples of the others, holding their pages together, and the pool is
brought together.

Random projections stand in for a model's queries, keys and values, and random
numbers for the verdict on drafts.  Every step is four calls and no read of a
device value: reserve pages and slots, append the new tokens' codes, attend, and
trim what was rejected or has finished.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import product_vq_kv_gb300 as vq

HQ, HKV, DIM, SUB, CENTROIDS, PAGE = 32, 8, 128, 8, 256, 16


class PagedCache:
    """The pool, the block tables and the lengths of a fixed number of request
    seats, on the device."""

    def __init__(self, seats: int, pages: int, max_blocks: int, device="cuda", dtype=torch.float16):
        ns = DIM // SUB
        self.codebooks = [torch.randn(HKV, CENTROIDS, SUB, device=device).to(dtype) for _ in range(2)]
        self.codes = torch.zeros(pages, 2, HKV, PAGE, ns, dtype=torch.uint8, device=device)
        self.table = torch.full((seats, max_blocks), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(pages, dtype=torch.int32, device=device)
        self.count = torch.tensor([pages], dtype=torch.int32, device=device)
        self.lens = torch.zeros(seats, dtype=torch.int32, device=device)

    def step(self, new_lens: torch.Tensor, rows: int, most: int, q, k, v):
        """Append `rows` packed new tokens, new_lens[r] of each request (at most
        `most`), and attend with them."""
        _, _, cu, slots = vq.vq_paged_reserve(self.lens, new_lens, self.free, self.count, self.table, PAGE, rows,
                                              lens_out=self.lens, free_count_out=self.count)
        kc, vc = self.codes[:, 0], self.codes[:, 1]
        vq.vq_paged_append(k, v, slots, *self.codebooks, kc, vc)
        return vq.vq_paged_attention(q, cu, self.lens, self.table, kc, vc, *self.codebooks, max_new=most, slots=slots)

    def keep(self, keep_lens: torch.Tensor):
        """Cut the requests to keep_lens tokens; their pages go back."""
        vq.vq_paged_trim(self.lens, keep_lens, self.table, PAGE, self.free, self.count, lens_out=self.lens,
                         free_count_out=self.count)


    def pools(self):
        return [self.codes]

    def fork(self, parents: torch.Tensor):
        """Seat d goes on where seat parents[d] stands; pages are shared."""
        self.lens, self.table, self.count, copies = vq.vq_paged_fork(self.lens, parents, self.table, PAGE, self.free, self.count)
        vq.vq_paged_copy(copies, self.pools())

    def compact(self):
        """Bring the held pages to the front of the pool."""
        moves = vq.vq_paged_compact(self.lens, self.table, PAGE, self.free, self.count, table_out=self.table,
                                    free_pages_out=self.free, free_count_out=self.count)[3]
        vq.vq_paged_copy(moves, self.pools())


class ScalarCache(PagedCache):
    """The same with 4-bit scalar codes and a scale a row."""

    def __init__(self, seats: int, pages: int, max_blocks: int, device="cuda", dtype=torch.float16):
        super().__init__(seats, pages, max_blocks, device, dtype)
        self.codes = torch.zeros(pages, 2, HKV, PAGE, DIM // 2, dtype=torch.uint8, device=device)
        self.scales = torch.zeros(pages, 2, HKV, PAGE, dtype=dtype, device=device)
        # for rows of root mean square one: sixteen steps over 2.7 of it either way
        self.centroids = torch.linspace(-2.7, 2.7, 16, device=device)
        self.signs = torch.randint(0, 2, (DIM,), device=device).float() * 2 - 1

    def step(self, new_lens: torch.Tensor, rows: int, most: int, q, k, v):
        _, _, cu, slots = vq.vq_paged_reserve(self.lens, new_lens, self.free, self.count, self.table, PAGE, rows,
                                              lens_out=self.lens, free_count_out=self.count)
        cache = (self.codes[:, 0], self.codes[:, 1], self.scales[:, 0], self.scales[:, 1])
        vq.vq_paged_scalar_append(k, v, slots, self.centroids, self.centroids, *cache, k_signs=self.signs)
        q = vq.vq_hadamard_rotate(q.reshape(-1, DIM), self.signs).reshape(q.shape).to(k.dtype)
        return vq.vq_paged_scalar_attention(q, cu, self.lens, self.table, *cache, self.centroids, self.centroids,
                                            max_new=most, slots=slots)

    def pools(self):
        return [self.codes, self.scales]


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--requests", type=int, default=12)
    ap.add_argument("--prompt", type=int, default=700, help="longest prompt")
    ap.add_argument("--answer", type=int, default=60, help="longest answer")
    ap.add_argument("--chunk", type=int, default=256, help="prompt tokens a step takes of a request")
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--scalar", action="store_true", help="4-bit scalar codes")
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    rng = torch.Generator().manual_seed(1)
    longest = args.prompt + args.answer + args.drafts + 1
    blocks = -(-longest // PAGE)
    cache = (ScalarCache if args.scalar else PagedCache)(args.requests, args.requests * blocks, blocks)

    def arrive():
        return {"prompt": int(torch.randint(1, args.prompt + 1, (1,), generator=rng)),
                "answer": int(torch.randint(1, args.answer + 1, (1,), generator=rng)), "held": 0}

    seats = [arrive() for _ in range(args.requests)]
    done = appended = 0
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.steps):
        new = []
        for s in seats:
            left = s["prompt"] - s["held"]
            new.append(min(left, args.chunk) if left > 0 else 1 + args.drafts)
        rows = sum(new)
        packed = torch.randn(rows, HQ + 2 * HKV, DIM, device="cuda", dtype=torch.float16)
        out = cache.step(torch.tensor(new, dtype=torch.int32, device="cuda"), rows, max(new), packed[:, :HQ],
                         packed[:, HQ:HQ + HKV], packed[:, HQ + HKV:])
        assert out.shape == (rows, HQ, DIM)
        keep = []
        for i, (s, n) in enumerate(zip(seats, new)):
            accepted = n
            if s["held"] >= s["prompt"]:
                accepted = 1 + int(torch.randint(0, args.drafts + 1, (1,), generator=rng))
            s["held"] += accepted
            appended += accepted
            if s["held"] >= s["prompt"] + s["answer"]:
                done += 1
                seats[i] = arrive()
            keep.append(seats[i]["held"])
        cache.keep(torch.tensor(keep, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start
    held = [s["held"] for s in seats]
    assert cache.lens.tolist() == held
    assert cache.count.item() == args.requests * blocks - sum(-(-h // PAGE) for h in held)
    # every other seat becomes a second sample of the seat before it
    cache.fork(torch.arange(args.requests, dtype=torch.int32, device="cuda") // 2 * 2)
    cache.compact()
    held = [held[i // 2 * 2] for i in range(args.requests)]
    assert cache.lens.tolist() == held
    used = sum(-(-h // PAGE) for h in held[::2]) + sum(h % PAGE != 0 for h in held[1::2])
    assert cache.count.item() == args.requests * blocks - used and cache.table.max().item() < used
    report = {"steps": args.steps, "tokens": appended, "finished": done, "held": sum(held),
              "ms_per_step": 1e3 * seconds / args.steps}
    print(report)
    return report


if __name__ == "__main__":
    main()
