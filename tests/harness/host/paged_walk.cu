// paged_walk.cu -- the paged attention's work split on the host: the layout and the
// walk of vq_pattn.cuh, block after block, as its kernels run them.

#include "vq_pattn.cuh"

namespace {

struct Walk {
    int64_t total, u0, u1;
    int32_t blocks, hx;
    int64_t j;
    int32_t r, at;
};

// What paged_plan leaves for block b: `threads` threads lay the items out.
Walk plan(const vqk::PagedArgs &a, const vqk::PagedLens &l, int threads, int64_t grid, int64_t b)
{
    Walk w{};
    for (int t = 0; t < threads; ++t) {
        int r0 = 0;
        w.total += vqk::PagedRun(a, t, threads).cost(a, l, &r0);
    }
    const int64_t all = w.total * a.hkv * a.gch, n = all < grid ? all : grid;
    w.blocks = (int32_t)n;
    if (b >= n) return w;
    w.u0 = vqk::part_of(b, all, n);
    w.u1 = vqk::part_of(b + 1, all, n);
    w.hx = (int32_t)(w.u0 / w.total);
    int64_t left = w.u0 % w.total;
    for (int t = 0; t < threads; ++t) {
        const vqk::PagedRun run(a, t, threads);
        int r0 = 0;
        const int64_t mine = run.cost(a, l, &r0);
        if (left < mine) {
            (void)run.locate(a, l, r0, left, &w.j, &w.r, &w.at);
            break;
        }
        left -= mine;
    }
    return w;
}

}  // namespace

// Segments of all blocks as rows of 10 numbers: block, head group, first token, tokens,
// position, k_lo + begin units, units, whole, slot, request; notes as rows of 7: block, token, head,
// heads, rows, first, last.  Returns segments; *n_notes the notes; -1 if they do not fit.
extern "C" int64_t paged_walk(const int32_t *cu, const int32_t *lens, int64_t requests, int64_t tokens,
                              int64_t max_blocks, int32_t page_shift, int32_t window, int32_t hkv, int32_t group,
                              int32_t gc, int32_t tile_tokens, int32_t item_cost, int32_t no_split, int32_t cls,
                              int32_t cls_tokens, int32_t threads, int64_t grid, int64_t room, int64_t *segments,
                              int64_t *notes, int64_t *n_notes)
{
    vqk::PagedArgs a{};
    a.tokens = tokens;
    a.requests = (int32_t)requests;
    a.max_blocks = (int32_t)max_blocks;
    a.page_shift = page_shift;
    a.window = window;
    a.hkv = hkv;
    a.group = group;
    a.gc = gc;
    a.gch = (group + gc - 1) / gc;
    a.tile_tokens = tile_tokens;
    a.item_cost = item_cost;
    a.no_split = no_split;
    a.cls = cls;
    a.cls_tokens = cls_tokens;
    a.items = tokens / tile_tokens + requests + 1;
    const vqk::PagedLens l{cu, lens, nullptr, a.requests, tile_tokens, tokens};
    int64_t count = 0;
    *n_notes = 0;
    for (int64_t b = 0; b < grid; ++b) {
        const Walk w = plan(a, l, threads, grid, b);
        if (b >= w.blocks) break;
        vqk::PagedCursor cur;
        cur.init(w, (int32_t)b);
        vqk::PagedSegment s;
        vqk::PagedNote note{};
        while (cur.next(a, w, l, s, note)) {
            if (count == room) return -1;
            const int64_t row[10] = {b,           s.hx,         s.it.tok0, s.it.ntok, s.it.pos0, s.it.k_lo + (int64_t)s.begin * vqk::kUnit,
                                     s.end - s.begin, s.whole, s.slot,    cur.r};
            for (int i = 0; i < 10; ++i) segments[count * 10 + i] = row[i];
            ++count;
        }
        if (note.rows) {
            const int64_t row[7] = {b, note.tok0, note.head0, note.gc, note.rows, note.first, note.last};
            for (int i = 0; i < 7; ++i) notes[*n_notes * 7 + i] = row[i];
            ++*n_notes;
        }
    }
    return count;
}
