// Drives the library's C ABI from a program whose host code (the library's
// included) is built with AddressSanitizer, so that the argument checks, the
// per-stream workspaces (growth, epochs, release), the static scratch and
// the dispatch tables run under it.
//
//   abi_asan host    argument checks and host-only calls (no GPU needed)
//   abi_asan device  the same, then scans, compactions, radix passes and CSR
//                    offsets on the GPU at sizes that grow each workspace
//                    several times, on two streams, with releases between
//
// Exit status 0 when every returned status and every checked output is as
// expected; AddressSanitizer ends the program with its own status on an error.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "dwpt_scan.h"
#include "dwpt_seq.h"

static int g_fail = 0;

#define EXPECT(cond)                                                          \
    do {                                                                      \
        if (!(cond)) {                                                        \
            std::fprintf(stderr, "%s:%d: expected %s\n", __FILE__, __LINE__, #cond); \
            ++g_fail;                                                         \
        }                                                                     \
    } while (0)

// The sequence operators' argument checks and workspace sizes.
static void seq_host_checks(uint32_t* buf)
{
    EXPECT(embedding_lookup(SEQ_F32, buf, 4, 0, buf, 4, 4, 4, 1.0f, buf, nullptr) == SCAN_OK);
    EXPECT(embedding_lookup(SEQ_F32, buf, 4, 4, buf, 4, 4, 4, 1.0f, buf, nullptr) == SCAN_ERR_INVALID);  // out over table
    EXPECT(embedding_grad(SEQ_F32, SEQ_F32, buf, 4, 4, buf, 4, 4, 4, 1.0f, 0, buf, nullptr, 0, nullptr) == SCAN_ERR_INVALID);
    EXPECT(embedding_grad_workspace(1000, 1000, 8) > 1000 * 4);
    EXPECT(causal_conv1d(nullptr, nullptr) == SCAN_ERR_INVALID);
    causal_conv1d_args_t c{};
    EXPECT(causal_conv1d(&c, nullptr) == SCAN_ERR_UNSUPPORTED);  // width 0
    EXPECT(causal_conv1d_grad_workspace(&c) == 0);
    selective_scan_args_t a{};
    EXPECT(selective_scan(&a, nullptr) == SCAN_ERR_UNSUPPORTED);  // no states
    a.states = 16;
    EXPECT(selective_scan(&a, nullptr) == SCAN_ERR_INVALID);  // no channels
    EXPECT(selective_scan_workspace(&a) == 0 && selective_scan_saved(&a) == 0);
    EXPECT(selective_scan_grad(nullptr, nullptr) == SCAN_ERR_INVALID);
    EXPECT(selective_scan_step(nullptr, nullptr) == SCAN_ERR_INVALID);
    gated_scan_args_t g{};
    EXPECT(gated_scan(&g, nullptr) == SCAN_ERR_INVALID);  // no channels
    EXPECT(gated_scan_workspace(&g) == 0 && gated_scan_saved(&g) == 0 && gated_scan_grad_workspace(nullptr) == 0);
    EXPECT(gated_scan_grad(nullptr, nullptr) == SCAN_ERR_INVALID && gated_scan_step(nullptr, nullptr) == SCAN_ERR_INVALID);
    int32_t* ints = reinterpret_cast<int32_t*>(buf);
    EXPECT(expert_split(ints, 4, 4, ints + 8, ints + 4, ints + 10, nullptr, 0, nullptr) == SCAN_ERR_INVALID);  // outputs overlap
    EXPECT(expert_split(ints, 5000, 4, ints, ints, ints, nullptr, 0, nullptr) == SCAN_ERR_INVALID);           // no workspace
    EXPECT(expert_split_workspace(100000, 64) >= 64 * 25 * 4);
    expert_dispatch_args_t d{};
    EXPECT(expert_dispatch(&d, nullptr) == SCAN_ERR_INVALID);
    expert_combine_args_t m{};
    m.choices = m.channels = 1;
    EXPECT(expert_combine(&m, nullptr) == SCAN_OK);  // no tokens
    EXPECT(expert_combine_grad(nullptr, nullptr) == SCAN_ERR_INVALID);
    sample_tokens_args_t t{};
    EXPECT(sample_tokens(&t, nullptr) == SCAN_ERR_INVALID);
}

static void host_checks()
{
    alignas(16) static uint32_t buf[64];
    void* odd = reinterpret_cast<char*>(buf) + 2;
    // argument checks that return before any device work
    EXPECT(scan_inclusive(SCAN_OP_ADD, SCAN_I32, nullptr, buf, 10, nullptr) == SCAN_ERR_INVALID);
    EXPECT(scan_inclusive(SCAN_OP_ADD, SCAN_I32, buf, nullptr, 10, nullptr) == SCAN_ERR_INVALID);
    EXPECT(scan_inclusive(SCAN_OP_ADD, SCAN_I32, odd, buf, 10, nullptr) == SCAN_ERR_INVALID);
    EXPECT(scan_exclusive(SCAN_OP_ADD, SCAN_I32, buf, buf + 1, 16, nullptr) == SCAN_ERR_INVALID);  // partial overlap
    EXPECT(scan_inclusive((scan_op_t)99, SCAN_I32, buf, buf, 1, nullptr) == SCAN_ERR_UNSUPPORTED);
    EXPECT(scan_inclusive(SCAN_OP_ADD, (scan_dtype_t)99, buf, buf, 1, nullptr) == SCAN_ERR_UNSUPPORTED);
    EXPECT(scan_inclusive(SCAN_OP_AFFINE, SCAN_F32, buf, buf, 1, nullptr) == SCAN_ERR_UNSUPPORTED);
    EXPECT(segmented_scan(SCAN_OP_ADD, SCAN_I32, buf, nullptr, buf, 10, 0, nullptr) == SCAN_ERR_INVALID);
    EXPECT(compact(SCAN_F32, buf, buf + 32, buf, 4, nullptr) == SCAN_ERR_INVALID);       // count inside the input
    EXPECT(compact(SCAN_F32, buf, buf + 32, buf + 33, 8, nullptr) == SCAN_ERR_INVALID);  // count inside the output
    EXPECT(compact(SCAN_F32, buf, buf + 32, nullptr, 8, nullptr) == SCAN_ERR_INVALID);
    EXPECT(radix_split(buf, nullptr, 16, 32, buf + 32, nullptr, nullptr) == SCAN_ERR_INVALID);  // shift past the key
    EXPECT(radix_split(buf, buf + 16, 16, 0, buf + 32, nullptr, nullptr) == SCAN_ERR_INVALID);  // values without output
    EXPECT(radix_split(buf, nullptr, 16, 0, buf + 8, nullptr, nullptr) == SCAN_ERR_INVALID);    // output overlaps keys
    EXPECT(csr_row_offsets(buf, 4, 3, nullptr, nullptr) == SCAN_ERR_INVALID);
    EXPECT(scan_noalloc(SCAN_OP_MAT3, SCAN_U32X9, buf, buf, (size_t)1 << 40, 0, nullptr) == SCAN_ERR_INVALID);
    seq_host_checks(buf);
    // strings and knobs
    for (int s = -1; s <= 7; ++s) EXPECT(std::strlen(scan_status_string((scan_status_t)s)) > 0);
    const size_t old = scan_set_small_n_max(123);
    EXPECT(scan_set_small_n_max(old) == 123);
    const int mode = scan_set_multi_tile_mode(2);
    EXPECT(scan_set_multi_tile_mode(mode) == 2);
    const uint32_t spin = scan_set_spin_limit(77);
    EXPECT(scan_set_spin_limit(spin) == 77);
}

#define HIPCHECK(x)                                                                       \
    do {                                                                                  \
        if ((x) != hipSuccess) {                                                          \
            std::fprintf(stderr, "%s:%d: %s failed\n", __FILE__, __LINE__, #x);           \
            std::exit(3);                                                                 \
        }                                                                                 \
    } while (0)

// One training pass of the sequence operators on a stream: tokens, table, convolution, scan and back.
static void seq_device_checks(hipStream_t st)
{
    const uint64_t b = 3, l = 150, rows = b * l;
    const uint32_t d = 72, n = 16, v = 100;
    std::vector<int32_t> tok(rows);
    for (uint64_t i = 0; i < rows; ++i) tok[i] = (int32_t)(i * 37 % 103) - 1;  // some outside the table
    std::vector<float> table(v * d, 0.25f), weight(d * 4, 0.5f), A(d * n, -1.0f), bc(rows * 2 * n, 0.5f);
    std::vector<void*> mem;
    const auto dev = [&](const void* src, size_t bytes) {
        void* p = nullptr;
        HIPCHECK(hipMalloc(&p, bytes));
        mem.push_back(p);
        if (src)
            HIPCHECK(hipMemcpy(p, src, bytes, hipMemcpyHostToDevice));
        else
            HIPCHECK(hipMemset(p, 0, bytes));
        return p;
    };
    const size_t big = rows * d * 4;
    void *dtok = dev(tok.data(), rows * 4), *dtab = dev(table.data(), v * d * 4), *e = dev(nullptr, big), *u = dev(nullptr, big);
    void *y = dev(nullptr, big), *dbc = dev(bc.data(), bc.size() * 4), *dw = dev(weight.data(), weight.size() * 4);
    EXPECT(embedding_lookup(SEQ_F32, dtok, 4, rows, dtab, d, v, d, 2.0f, e, st) == SCAN_OK);
    causal_conv1d_grad_args_t cg{};
    causal_conv1d_args_t& c = cg.args;
    c.width = 4;
    c.activation = SEQ_ACT_SILU;
    c.rows = rows;
    c.seqs = b;
    c.channels = d;
    c.x = e;
    c.x_stride = c.y_stride = d;
    c.weight = dw;
    c.y = u;
    EXPECT(causal_conv1d(&c, st) == SCAN_OK);
    selective_scan_grad_args_t sg{};
    selective_scan_args_t& a = sg.args;
    a.rows = rows;
    a.seqs = b;
    a.channels = d;
    a.states = n;
    a.groups = 1;
    a.delta_softplus = 1;
    a.x = a.delta = u;
    a.x_stride = a.delta_stride = a.y_stride = d;
    a.A = (const float*)dev(A.data(), A.size() * 4);
    a.B = dbc;
    a.C = (const float*)dbc + n;
    a.b_stride = a.c_stride = 2 * n;
    a.y = y;
    a.saved = (float*)dev(nullptr, selective_scan_saved(&a) * 4);
    a.workspace_bytes = selective_scan_workspace(&a);
    a.workspace = dev(nullptr, a.workspace_bytes);
    EXPECT(selective_scan(&a, st) == SCAN_OK);
    sg.dy = y;
    sg.dx = dev(nullptr, big);
    sg.ddelta = dev(nullptr, big);
    sg.dB = dev(nullptr, rows * n * 4);
    sg.dC = dev(nullptr, rows * n * 4);
    sg.dy_stride = sg.dx_stride = sg.ddelta_stride = d;
    sg.db_stride = sg.dc_stride = n;
    sg.dA = (float*)dev(nullptr, A.size() * 4);
    a.workspace_bytes = selective_scan_grad_workspace(&sg);
    a.workspace = dev(nullptr, a.workspace_bytes);
    EXPECT(selective_scan_grad(&sg, st) == SCAN_OK);
    cg.dy = sg.dx;
    cg.dx = dev(nullptr, big);
    cg.dy_stride = cg.dx_stride = d;
    cg.dweight = (float*)dev(nullptr, weight.size() * 4);
    cg.workspace_bytes = causal_conv1d_grad_workspace(&c);
    cg.workspace = dev(nullptr, cg.workspace_bytes);
    EXPECT(causal_conv1d_grad(&cg, st) == SCAN_OK);
    const size_t need = embedding_grad_workspace(rows, v, d);
    EXPECT(embedding_grad(SEQ_F32, SEQ_F32, dtok, 4, rows, cg.dx, d, v, d, 2.0f, 0, dtab, dev(nullptr, need), need, st) == SCAN_OK);
    HIPCHECK(hipStreamSynchronize(st));
    float first = -1.0f;  // u[0] = silu(e[0] * 0.5): token -1 is a row of zeros
    HIPCHECK(hipMemcpy(&first, u, 4, hipMemcpyDeviceToHost));
    EXPECT(first == 0.0f);
    for (void* p : mem) HIPCHECK(hipFree(p));
}

// A recurrent layer with experts and the next tokens on a stream: gated scan and back, a split of every row to two
// experts, their rows out and in, and a sampled channel per row.
static void recurrent_device_checks(hipStream_t st)
{
    const uint32_t rows = 400, seqs = 2, d = 72, e = 5, k = 2;
    std::vector<int32_t> experts(rows * k);
    for (uint32_t i = 0; i < rows * k; ++i) experts[i] = (int32_t)(i * 7 % (e + 1));  // some of no expert
    std::vector<float> ones(rows * d, 1.0f), rate(d, -0.5f);
    std::vector<void*> mem;
    const auto dev = [&](const void* src, size_t bytes) {
        void* p = nullptr;
        HIPCHECK(hipMalloc(&p, bytes));
        mem.push_back(p);
        if (src)
            HIPCHECK(hipMemcpy(p, src, bytes, hipMemcpyHostToDevice));
        else
            HIPCHECK(hipMemset(p, 0, bytes));
        return p;
    };
    const size_t big = rows * d * 4;
    gated_scan_grad_args_t g{};
    gated_scan_args_t& a = g.args;
    a.rows = rows;
    a.seqs = seqs;
    a.channels = d;
    a.x = a.decay_gate = a.input_gate = dev(ones.data(), big);
    a.x_stride = a.decay_stride = a.input_stride = a.y_stride = d;
    a.rate = (const float*)dev(rate.data(), d * 4);
    a.y = dev(nullptr, big);
    a.saved = (float*)dev(nullptr, gated_scan_saved(&a) * 4);
    a.workspace_bytes = gated_scan_workspace(&a);
    a.workspace = dev(nullptr, a.workspace_bytes);
    EXPECT(gated_scan(&a, st) == SCAN_OK);
    g.dy = a.y;
    g.dx = dev(nullptr, big);
    g.ddecay_gate = dev(nullptr, big);
    g.dinput_gate = dev(nullptr, big);
    g.dy_stride = g.dx_stride = g.ddecay_stride = g.dinput_stride = d;
    g.drate = (float*)dev(nullptr, d * 4);
    a.workspace_bytes = gated_scan_grad_workspace(&a);
    a.workspace = dev(nullptr, a.workspace_bytes);
    EXPECT(gated_scan_grad(&g, st) == SCAN_OK);

    int32_t *choices = (int32_t*)dev(experts.data(), experts.size() * 4), *offsets = (int32_t*)dev(nullptr, (e + 1) * 4);
    int32_t *places = (int32_t*)dev(nullptr, rows * k * 4), *source = (int32_t*)dev(nullptr, rows * k * 4);
    const size_t need = expert_split_workspace(rows * k, e);
    EXPECT(need == 0);  // one chunk of choices
    EXPECT(expert_split(choices, rows * k, e, offsets, places, source, nullptr, 0, st) == SCAN_OK);
    expert_dispatch_args_t x{};
    x.tokens = rows;
    x.rows = rows * k;
    x.choices = k;
    x.channels = d;
    x.places = places;
    x.used = offsets + e;
    x.x = a.y;
    x.out = dev(nullptr, k * big);
    x.x_stride = x.out_stride = d;
    EXPECT(expert_dispatch(&x, st) == SCAN_OK);
    expert_combine_args_t c{};
    c.tokens = rows;
    c.rows = rows * k;
    c.choices = k;
    c.channels = d;
    c.places = places;
    c.y = x.out;
    c.out = dev(nullptr, big);
    c.y_stride = c.out_stride = d;
    EXPECT(expert_combine(&c, st) == SCAN_OK);
    expert_combine_grad_args_t q{};
    q.tokens = rows;
    q.rows = rows * k;
    q.choices = k;
    q.channels = d;
    q.places = places;
    q.used = offsets + e;
    q.dout = c.out;
    q.y = x.out;
    q.dy = dev(nullptr, k * big);
    q.dout_stride = q.y_stride = q.dy_stride = d;
    q.dweights = (float*)dev(nullptr, rows * k * 4);
    EXPECT(expert_combine_grad(&q, st) == SCAN_OK);
    sample_tokens_args_t t{};
    t.token_bytes = 4;
    t.rows = rows;
    t.n = d;
    t.logits = c.out;
    t.logits_stride = d;
    t.uniform = (const float*)dev(nullptr, rows * 4);
    t.temperature = t.top_p = 1.0;
    t.tokens = source;
    EXPECT(sample_tokens(&t, st) == SCAN_OK);
    HIPCHECK(hipStreamSynchronize(st));
    int32_t first = -1, used = 0;  // equal channels and a random number of 0: token 0
    HIPCHECK(hipMemcpy(&first, source, 4, hipMemcpyDeviceToHost));
    HIPCHECK(hipMemcpy(&used, offsets + e, 4, hipMemcpyDeviceToHost));
    int32_t want = 0;
    for (int32_t v : experts) want += v < (int32_t)e;
    EXPECT(first == 0 && used == want);
    for (void* p : mem) HIPCHECK(hipFree(p));
}

static void device_checks()
{
    int ndev = 0;
    HIPCHECK(hipGetDeviceCount(&ndev));
    EXPECT(ndev >= 1);
    hipStream_t s[2];
    HIPCHECK(hipStreamCreate(&s[0]));
    HIPCHECK(hipStreamCreate(&s[1]));
    const size_t nmax = (size_t)1 << 24;
    int32_t *x, *y;
    uint32_t *cnt, *keys, *kout, *rowp;
    uint8_t* heads;
    HIPCHECK(hipMalloc(&x, nmax * 4));
    HIPCHECK(hipMalloc(&y, nmax * 4));
    HIPCHECK(hipMalloc(&cnt, 4));
    HIPCHECK(hipMalloc(&keys, nmax * 4));
    HIPCHECK(hipMalloc(&kout, nmax * 4));
    HIPCHECK(hipMalloc(&heads, nmax));
    HIPCHECK(hipMalloc(&rowp, ((size_t)1 << 16) * 4 + 4));
    std::vector<int32_t> hx(nmax);
    for (size_t i = 0; i < nmax; ++i) hx[i] = (int32_t)(i % 7) - 3;
    std::vector<uint32_t> hk(nmax);
    for (size_t i = 0; i < nmax; ++i) hk[i] = (uint32_t)(i * 2654435761u) % (1u << 16);
    HIPCHECK(hipMemcpy(x, hx.data(), nmax * 4, hipMemcpyHostToDevice));
    HIPCHECK(hipMemcpy(keys, hk.data(), nmax * 4, hipMemcpyHostToDevice));
    HIPCHECK(hipMemset(heads, 0, nmax));
    for (int round = 0; round < 2; ++round) {
        // sizes that grow every workspace several times; both streams; every kernel path
        for (size_t n : {(size_t)1, (size_t)1000, (size_t)20000, (size_t)1 << 20, nmax}) {
            for (int mode : {0, 1, 2, 3}) {
                const int old = scan_set_multi_tile_mode(mode);
                hipStream_t st = s[(n + mode) % 2];
                EXPECT(scan_inclusive(SCAN_OP_ADD, SCAN_I32, x, y, n, st) == SCAN_OK);
                EXPECT(scan_exclusive(SCAN_OP_MAX, SCAN_I32, x, y, n, st) == SCAN_OK);
                EXPECT(segmented_scan(SCAN_OP_ADD, SCAN_I32, x, heads, y, n, 0, st) == SCAN_OK);
                EXPECT(compact(SCAN_I32, x, y, cnt, n, st) == SCAN_OK);
                scan_set_multi_tile_mode(old);
            }
            EXPECT(scan_noalloc(SCAN_OP_ADD, SCAN_I32, x, y, n, 1, s[0]) == SCAN_OK);
            EXPECT(radix_split(keys, nullptr, n, 8, kout, nullptr, s[1]) == SCAN_OK);
            if (n >= 2)
                EXPECT(radix_split(keys, keys + n / 2, n / 2, 0, kout, kout + n / 2, s[0]) == SCAN_OK);
            EXPECT(csr_row_offsets(kout, n, 1u << 16, rowp, s[1]) == SCAN_OK);
            HIPCHECK(hipDeviceSynchronize());
            EXPECT(scan_get_device_error(s[0]) == SCAN_OK);
            EXPECT(scan_get_device_error(s[1]) == SCAN_OK);
            // the last inclusive sum over the full size, against the host
            EXPECT(scan_inclusive(SCAN_OP_ADD, SCAN_I32, x, y, n, s[0]) == SCAN_OK);
            HIPCHECK(hipStreamSynchronize(s[0]));
            int32_t last = 0;
            HIPCHECK(hipMemcpy(&last, y + (n - 1), 4, hipMemcpyDeviceToHost));
            int64_t want = 0;
            for (size_t i = 0; i < n; ++i) want += hx[i];
            EXPECT(last == (int32_t)want);
        }
        EXPECT(scan_release_workspace() == SCAN_OK);
    }
    for (int i = 0; i < 2; ++i) seq_device_checks(s[i]);
    for (int i = 0; i < 2; ++i) recurrent_device_checks(s[i]);
    HIPCHECK(hipFree(x));
    HIPCHECK(hipFree(y));
    HIPCHECK(hipFree(cnt));
    HIPCHECK(hipFree(keys));
    HIPCHECK(hipFree(kout));
    HIPCHECK(hipFree(heads));
    HIPCHECK(hipFree(rowp));
    HIPCHECK(hipStreamDestroy(s[0]));
    HIPCHECK(hipStreamDestroy(s[1]));
}

int main(int argc, char** argv)
{
    const bool device = argc > 1 && std::strcmp(argv[1], "device") == 0;
    host_checks();
    if (device) device_checks();
    std::printf("abi_asan %s: %d failed checks\n", device ? "device" : "host", g_fail);
    return g_fail ? 1 : 0;
}
