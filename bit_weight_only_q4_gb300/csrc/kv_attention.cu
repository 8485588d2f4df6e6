// Host side of the attention over the paged cache: choice of kernel, workspace, launches.
// The kernels: kv_attention_few.cuh, kv_attention_many.cu; what they compute and how work
// is dealt out: kv_attention.cuh.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "kv_attention.cuh"

namespace q4 {

static std::atomic<int> g_give_up{-1}, g_give_up_tiles{0};

void kv_set_give_up(int cta, int tiles)
{
    g_give_up_tiles.store(tiles);
    g_give_up.store(cta);
}

struct KvPlan {
    KvKernel k;
    int row_tiles, grid;
    int64_t rows;
};

constexpr int kMaxGrid = Q4_KV_COUNTER_BYTES / 4;          // a counter for each CTA

static KvPlan kv_plan(const DeviceInfo &dev, const KvCacheDesc &c, int64_t rows)
{
    KvPlan t = {};
    t.rows = rows;
    // More rows than the few-row kernel's tile of 16: it would read and decode every token once
    // per 16 rows.  16,384 to 65,536 cached tokens, 8 key heads (us, few / many): 20 or 32 rows
    // 64 - 92 / 56 - 69 (int8 and int4, heads of 128), 53 - 59 / 43 - 61 (of 64); 48 rows
    // 73 - 113 / 44 - 72; 64 rows 91 - 175 / 45 - 74.
    if (rows > 16)
        t.k = kv_many_kernel(dev, c.format, c.head_dim);
    else
        t.k = c.format == Q4_CACHE_INT8 ? kv_few_kernel_int8(dev, c.head_dim, (int)rows)
                                        : kv_few_kernel_int4(dev, c.head_dim, (int)rows);
    t.row_tiles = (int)((rows + t.k.tile - 1) / t.k.tile);
    t.grid = dev.sms < kMaxGrid ? dev.sms : kMaxGrid;
    return t;
}

// Workspace: counters, at the same place for calls of every shape (they have to be zero when
// a call begins, and whatever else lies there need not be), then the pieces of the (one or
// two) launches, which follow one another, then the prefix's results.
struct KvWorkspace {
    size_t piece_o, piece_ml, prefix_o, prefix_ml, total;
};

static KvWorkspace kv_workspace(const KvCacheDesc &c, const KvPlan *plans, int n, int64_t prefix_rows)
{
    KvWorkspace w = {};
    auto take = [&](size_t bytes) {
        const size_t at = w.total;
        w.total += (bytes + 255) / 256 * 256;
        return at;
    };
    size_t piece_rows = 0;
    for (int i = 0; i < n; ++i)
        piece_rows = std::max(piece_rows, (size_t)2 * plans[i].grid * plans[i].k.tile);
    take(Q4_KV_COUNTER_BYTES);
    w.piece_o = take(piece_rows * c.head_dim * 4);
    w.piece_ml = take(piece_rows * 2 * 4);
    w.prefix_o = take((size_t)prefix_rows * c.heads * c.head_dim * 4);
    w.prefix_ml = take((size_t)prefix_rows * c.heads * 2 * 4);
    return w;
}

// One launch over the sequences' own tokens; before it, with a shared prefix, one over the
// prefix for the rows of all sequences, whose results the second takes up.
static int kv_plans(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens, int q_heads, int prefix_len,
                    KvPlan (&plans)[2])
{
    const int64_t rows = (int64_t)tokens * (q_heads / c.heads);
    plans[0] = kv_plan(dev, c, rows);
    if (prefix_len <= 0)
        return 1;
    plans[1] = kv_plan(dev, c, rows * batch);
    return 2;
}

size_t kv_attention_workspace_bytes(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens,
                                    int q_heads, int prefix_len)
{
    KvPlan plans[2];
    const int n = kv_plans(dev, c, batch, tokens, q_heads, prefix_len, plans);
    return kv_workspace(c, plans, n, n == 2 ? plans[1].rows : 0).total;
}

// Lets a kernel have the shared memory that its launches ask for, once per context and
// larger size (the call costs about as much as a launch).
static q4_status kv_allow_smem(const KvKernel &k)
{
    struct Set {
        const void *fn;
        void *ctx;
        size_t bytes;
    };
    static std::mutex mu;
    static Set sets[16];
    void *ctx = current_context();
    std::lock_guard<std::mutex> lock(mu);
    Set *at = nullptr;
    for (Set &s : sets)
        if (s.fn == k.fn || (!s.fn && !at)) {
            at = &s;
            if (s.fn)
                break;
        }
    if (at && at->fn == k.fn && ctx && at->ctx == ctx && at->bytes >= k.smem)
        return Q4_OK;
    cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(attention kernel)");
    if (at)
        *at = Set{k.fn, ctx, k.smem};
    return Q4_OK;
}

static q4_status kv_tile_launch(const KvPlan &plan, KvTileParams &p, cudaStream_t st, bool pdl)
{
    p.rows = (int)plan.rows;
    p.row_tiles = plan.row_tiles;
    p.stages = plan.k.stages;
    q4_status s = kv_allow_smem(plan.k);
    if (s != Q4_OK)
        return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.grid);
    cfg.blockDim = dim3((unsigned)plan.k.threads);
    cfg.dynamicSmemBytes = plan.k.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    void *args[] = {&p};
    cudaError_t e = cudaLaunchKernelExC(&cfg, plan.k.fn, args);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of the attention kernel");
}

q4_status launch_kv_attention(const DeviceInfo &dev, const KvCacheDesc &c, const KvAttnArgs &a, cudaStream_t st,
                              bool pdl)
{
    KvPlan plans[2];
    const int n = kv_plans(dev, c, a.batch, a.tokens, a.q_heads, a.prefix_len, plans);
    const KvWorkspace w = kv_workspace(c, plans, n, n == 2 ? plans[1].rows : 0);
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    auto at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };
    KvTileParams p = {};
    p.cache = KvCache{c.data, c.pages, c.heads, c.page_shift, (1 << c.page_shift) / KV_BLOCK};
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.lengths = a.lengths;
    p.tokens = a.tokens;
    p.group = a.q_heads / c.heads;
    p.by_tokens = KvDivisor((uint32_t)p.tokens);
    p.by_group = KvDivisor((uint32_t)p.group);
    p.all_rows = (int)(plans[0].rows * a.batch);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.err = device_error_flags();
    p.give_up = g_give_up.load();
    p.give_up_tiles = g_give_up_tiles.load();
    p.tickets = reinterpret_cast<unsigned *>(ws);
    p.piece_o = at(w.piece_o);
    p.piece_ml = at(w.piece_ml);
    // A prefix's results lie in the workspace between the two launches: no launch of another host
    // thread's call, which may use the same stream and workspace, may come in between.
    static std::mutex launches;
    std::lock_guard<std::mutex> lock(launches);
    q4_status s;
    if (n == 2) {
        KvTileParams f = p;
        f.table = a.prefix_pages;
        f.cap = a.prefix_len;
        f.seqs = 1;
        f.prefix_len = a.prefix_len;
        f.prefix_out_o = at(w.prefix_o);
        f.prefix_out_ml = at(w.prefix_ml);
        if ((s = kv_tile_launch(plans[1], f, st, pdl)) != Q4_OK)
            return s;
        p.prefix_in_o = f.prefix_out_o;
        p.prefix_in_ml = f.prefix_out_ml;
    }
    p.table = a.table;
    p.table_width = a.table_width;
    p.cap = (int64_t)a.table_width << c.page_shift;
    p.seqs = a.batch;
    return kv_tile_launch(plans[0], p, st, pdl);
}

}  // namespace q4
